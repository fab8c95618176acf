// The selective scan over whole sequences, by chunks of 128 tokens on the tcgen05 tensor cores.
//
// Per head, S [p][n], a token does  S <- exp(g) S + (dt x) B^T,  o = S C + D x,  g = dt A.
// Over a chunk from state S0, with G_t the sum of g up to token t, unrolling gives
//     O   = diag(exp G) C S0^T + M X + D X,   M_ts = exp(G_t - G_s) dt_s <C_t, B_s> for s <= t
//     S_L = exp(G_L) S0 + X^T diag(dt exp(G_L - G)) B
// All factors are exp of sums of g over s + 1 .. t, so at most 1: no decay is too strong.  G is kept
// in fixed point, 64 bits with 2^-40 the last one, so that its differences are exact, also after a token
// that empties the state (g log2 e is taken as between -160 and 160; 2^-160 is 0 in float32).
//
// Precision.  x, B and C are bf16 and go to the tensor cores as they were loaded.  The computed
// operands (S0, M, the weighted X) are split into two bf16 parts, 16 bits, which leave 2^-18 of them.  D x, the
// largest part of most outputs, is added in float32 as x's row gives way to them: with D in M's diagonal the error of float32
// outputs was 2.2e-6 instead of 1.0e-6 (rms, against float32 torch).  It takes one more read of x's tile a chunk: 8 x 4,096
// tokens of 64 heads of 64 x 128 258 -> 264 us, with bf16 states 315 -> 331, with float32 outputs, two passes over the
// tile, 278 -> 309; 1 x 16,383 of 16 heads of 128 x 128, float32 outputs, 142 -> 146, with bf16 states 161 -> 164.
// Sums and states are float32; the states stay in tensor memory from chunk to chunk.  Where they are stored as
// bf16 the weighted X has three parts (W3): an error of 1.1e-6 of a state's size, as two leave, rounds 1.4 of 1,000
// entries to the other neighbour, 2^-8 of them away, and the next call's outputs show it; three leave 0.07 of
// 1,000 (float32 torch operations about as many).  x has two stages then, and U is taken by 64 columns: 8 x 4,096 tokens
// 331 us instead of 264, 1 x 16,383 of 16 heads 164 instead of 146.  (U's first two parts at 128 columns and a wait before the
// third: 1 and 3 us more.)
//
// The unit of work is 64 rows (of p) of one (sequence, head).  A CTA an SM takes its share of all chunks, unit
// after unit, and its roles run on from one unit into the next.  Its warps:
//   scores (0-7)    row t of M from C B^T, in tensor memory, back in its place, 16 columns at a time: warps 0-3 and
//                   4-7 half of each diagonal block of 32 x 32 and half of what lies below it
//   states (8-15)   column j of S, 32 of its 64 values a thread; two bf16 parts of it for the next chunk's C S0^T
//   steps (16-19)   row s of the weighted X
//   outputs (20-23) row t of O
//   issue (24)      the MMAs;  scalars (25, 26) G and dt of each token, every other chunk;  loads (27) TMA,
//                   and what the next unit is
// Four products a chunk, all of M = 128:
//     C B^T          N = 128 (s), K = n
//     U = B^T [Xh Xl]    N = 128, K = 128 (s); the halves add up (W3: N = 64 each, the third onto the second)
//     C [Sh Sl]      N = 128, K = n; the halves add up
//     [Mh Ml] X      N = 64, K = 2 x 128 (s), M from tensor memory
// M's decays take one 2^x a row and not one an entry: below its diagonal blocks of 32 x 32 they are products of two
// factors at most 1 that meet at the border before row t's block, in them running products of single
// tokens' decays (at most 16, from the diagonal or from the block's middle on).
//
// Bound by shared memory: of a chunk's 4,700 cycles (8 x 4,096 tokens of 64 heads of 64 x 128: 264 us, 108 chunks an SM)
// its reads and writes take 3,700 (the products' operands 1,800, TMA 640, the two parts of S and of the weighted X as they
// are written and x as it is read twice 770, the outputs 260, the factors the rest) and more with the conflicts between them; the tensor
// cores are busy for 2,080, the issue slots for half.  Its inputs, outputs and states alone, at the copy rate, would take
// 88 us.  What brought it there, us: 635 at first; 555 with MMAs issued under elect; 347 with every role's code
// small enough for the instruction cache and next to no spills; 335 with S in tensor memory and a third stage of x; 283 with
// equal stretches (512 units are 3.4 rounds of 152); 266 with running products of decays, sums in fixed point and
// outputs by TMA, 271 with D x in float32 (in a plain loop of calls 258 and 264).  A unit's start and end cost about 3 us, a launch 8.
//
// Values that are not finite.  In a product over the tokens of a chunk a zero coefficient does not keep a
// NaN or an infinity of a later token away from an earlier one, as the formulas do.  A row of S that
// meets one in x, B or dt has an entry that is not finite from then on, so such rows show in the
// unit's last state: they run through its tokens once more, one by one in float32.
//
// Shares.  All chunks of a call stand in one line, sequence after sequence and unit after unit, and each CTA
// takes an equal stretch of it.  A unit that a border cuts goes on in the next CTA from the float32
// state that the first left in the workspace.  A CTA begins with the unit that its end cuts, so that the
// next CTA, which ends with that unit's rest, finds the state there.  A unit longer than a stretch runs through several
// CTAs that have nothing else to do and do wait, one for the other: a call of one long sequence among short ones takes as
// long as that one's chunks in a row, 2.1 us each (16 heads, 32,768 tokens and nine times 100, 572 us; the long
// one alone, in segments, 145).  CTAs take their stretches in the order in
// which they start: the one that another waits for has started before it.  (Without a workspace no unit is cut.)
//
// Few units leave SMs idle, so long sequences are then cut into segments of whole chunks: TRANS runs each
// segment but the last from zero, without outputs; ssm_join_kernel chains the segments' states (S <- d S + that, d
// the segment's decay); then the ordinary kernel runs all segments as units of their own.
#include "chunk_common.cuh"
#include "device_common.cuh"
#include "gdn_internal.h"
#include "ssm_chunk.h"
#include "ssm_scalars.cuh"

#include <algorithm>
#include <cmath>

namespace wkv7 {
namespace {

constexpr int kL = 128;
// Warps, each role's first (scores begin at 0).  28 leave 72 registers a thread, which the roles are written for: a
// value spilled goes through an L1 that shared memory leaves almost nothing of.  (At d_state 128 the compiler spills 28 bytes
// a thread, 36 with float32 outputs, 44 in the first pass of segments; at 64 at most 16.)
constexpr int kStateWarp = 8, kStepWarp = 16, kOutWarp = 20, kIssueWarp = 24, kScalWarp = 25, kScalWarps = 2, kLoadWarp = 27;
constexpr int kThreads = 28 * 32;
constexpr int kStages = 2, kScal = 4;
constexpr int kTasks = 4;    // units known ahead
constexpr int kUnitCost = 2; // what a unit's start and end cost, in chunks

// Tensor-memory columns (512 allocated): C B^T, then M in its place (of each 16 columns, 8 of the
// high parts and 8 of the low ones, K elements 2c, 2c + 1 in a column); M X; C S0 in two halves; U in two
// halves; S, column j in lane j.
constexpr uint32_t kColM = 0, kColY = 128, kColCS = 192, kColU = 320, kColS = 448;

constexpr uint32_t kTile = 16384;  // 128 rows of 128 bytes, 128-byte swizzle

// A chunk's per-token values: G in fixed point, in units of log 2, dt and exp g; after them exp(G_L).
struct Scal {
    long long g[kL];
    float dt[kL];
    float after[kL];  // exp g of the token after this one (of a block's last: not used)
    float decay, pad[3];
};

// A unit, or the part of one that a CTA takes: `len` tokens from t0 on, where its state comes from (null: zeros) and
// goes to (null: nowhere), and which CTAs' parts it goes on from and is followed by (-1: none).
struct Task {
    int chunks, len, t0, h, row0;
    int from_bf16, to_bf16;
    int after, signal;
    long long mark;  // (TRANS) [unit][segment], for the segment's decay
    const void *from;
    void *to;
};
// A place in the line of all chunks: `chunk` of unit `unit` of sequence (or segment) vs.
struct Spot {
    int vs, unit, chunk;
};

// (W3: the weighted X in three parts, in the place of x's third stage)
template <int NS, bool W3>
struct Smem {
    static constexpr int kStagesX = W3 ? 2 : 3, kPartsW = W3 ? 3 : 2;
    static constexpr uint32_t kState = NS / 64 * kTile;     // a tile of B or C
    static constexpr uint32_t oC = 0;                       // per stage
    static constexpr uint32_t oX = oC + kStages * kState;   // per stage; the outputs pass through it
    static constexpr uint32_t oB = oX + kStagesX * kTile;
    static constexpr uint32_t oW = oB + kState;             // the weighted X, high parts first
    static constexpr uint32_t oS = oW + kPartsW * kTile;          // S: rows j of 64 (p), high parts then low
    static constexpr uint32_t kS = NS * 128;
    static constexpr uint32_t oScal = oS + 2 * kS;
    static constexpr uint32_t oV = oScal + kScal * sizeof(Scal);  // per scores warp: the border factors of its columns
    static constexpr uint32_t oBar = oV + 8 * 64 * 4;
    static constexpr uint32_t kBars = 2 * kStages + 2 * kStagesX + 1 + 2 * kScal + 2 * kTasks + 10;
    static constexpr uint32_t oHold = oBar + kBars * 8;
    static constexpr uint32_t oRedo = oHold + 32;  // per row: marked (see the file's header)
    static constexpr uint32_t oTask = oRedo + 64;
    static constexpr uint32_t kBytes = oTask + kTasks * sizeof(Task);
};

struct Maps {
    CUtensorMap x, b, c, o;
};

// A cut sequence's segments: `tokens` each (a multiple of 128; 0: not cut).  state[unit][n][64][NS]: what
// segment j alone leaves from zero at j + 1, after the join the state that segment j starts from at j;
// decay, done [unit][n - 1]: written when a segment is (done is cleared before); lost [unit]: one was not, and then
// the unit keeps its slot's state.
struct Segments {
    int tokens, n;
    float *state, *decay;
    int *done, *lost;
};
// Where units may be cut: `carry` [CTA][64][NS] the states handed on, `done` [CTA] whether they are there, `drawn` the
// CTAs that have started (both cleared before).  carry null: nowhere.
struct Shares {
    float *carry;
    unsigned *done, *drawn;
};

__device__ __forceinline__ F2 pair_of(uint32_t bf16x2) { return f2_bf16(bf16x2); }

// x = hi + mid + lo up to 2^-27 of it, bf16 each.
__device__ __forceinline__ void split3(F2 x, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    float a, b;
    unpack(x, a, b);
    hi = pack_bf16_rn(a, b);
    split2(fma2(pair_of(hi), f2(-1.f, -1.f), x), mid, lo);
}

// A wait that ends: with the phase, when another role has given up, or after the limit.  (Short, for the
// instruction cache's sake: it is at two dozen places.)
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, volatile int *flag, long long limit) {
    if (mbar_try_wait(bar, parity)) return;
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait_sleep(bar, parity, 2000u)) {
        if (*flag) return;
        if (clock64() - t0 > limit) *flag = 1;
    }
}
// 2^x of x in fixed point.
__device__ __forceinline__ float ex2_fixed(long long x) { return ex2_approx(__ll2float_rn(x) * 0x1p-40f); }

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __int_as_float(0x7f800000); }

// One lane of a converged warp.  (MMAs issued under it take the tensor core's time, 65 cycles for 128 x 128 x
// 16 and 33 for 128 x 64 x 16; under a comparison of lane numbers every operand goes through a loop over
// the lanes, and a chunk's 40 took 6,000 cycles instead of 2,100.)
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;}" : "=r"(p));
    return p != 0;
}

// D (+)= A B^T, `N` slices of 16 along K whose descriptors are a_step and b_step bytes apart.
template <int N>
__device__ __forceinline__ void umma_slices(uint32_t d, uint64_t a, uint32_t a_step, uint64_t b, uint32_t b_step, uint32_t idesc,
                                            bool accumulate) {
#pragma unroll
    for (int k = 0; k < N; ++k)
        umma_bf16(d, a + k * (a_step >> 4), b + k * (b_step >> 4), idesc, accumulate || k > 0 ? 1u : 0u);
}

// A unit's tokens for four of its rows (those in `mine`), one by one in float32, by a warp.  Rare, so written to be small.
template <int NS>
__device__ __noinline__ void run_by_token(const SsmRunArgs &p, const Task &t, int r0, uint32_t mine, bool outputs) {
    constexpr int R = 4, C = NS / 32;
    const int lane = threadIdx.x & 31;
    const int at = r0 * NS + lane * C;
    float s[R][C];
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int x = at + m * NS + c;
            s[m][c] = !t.from ? 0.f
                      : t.from_bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(t.from)[x]) << 16)
                                    : __ldcg(static_cast<const float *>(t.from) + x);
        }
    const int g = t.h / (p.lv.heads / p.lv.groups);
    const float d = p.in.d ? __ldg(p.in.d + t.h) : 0.f;
#pragma unroll 1
    for (int k = 0; k < t.len; ++k) {
        const long long row = static_cast<long long>(t.t0) + k;
        const StepScalars sc = step_scalars(p.in, t.h, load_dt(p.in, row, t.h));
        float b[C], c[C];
#pragma unroll
        for (int e = 0; e < C; ++e) {
            b[e] = load1<true>(p.in.b, row * p.in.b_stride + static_cast<long long>(g) * NS + lane * C + e);
            c[e] = load1<true>(p.in.c, row * p.in.c_stride + static_cast<long long>(g) * NS + lane * C + e);
        }
#pragma unroll
        for (int m = 0; m < R; ++m) {
            const int i = t.row0 + r0 + m;
            const float x = load1<true>(p.in.x, row * p.in.x_stride + static_cast<long long>(t.h) * p.lv.p + i);
            const float u = __fmul_rn(sc.dt, x);
            float y = 0.f;
#pragma unroll
            for (int e = 0; e < C; ++e) {
                s[m][e] = __fmaf_rn(sc.a, s[m][e], __fmul_rn(u, b[e]));
                y = fmaf(s[m][e], c[e], y);
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
            if (outputs && lane == 0 && (mine >> m & 1))
                store_out(p.in.o, p.in.o_bf16, (static_cast<size_t>(row) * p.lv.heads + t.h) * p.lv.p + i, p.in.d ? fmaf(d, x, y) : y);
        }
    }
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (t.to && (mine >> m & 1)) store_out(t.to, t.to_bf16, at + m * NS + c, s[m][c]);
}

// A sequence's (or segment's) tokens; no chunks where there is nothing to do.
struct Span {
    int slot, t0, t1, chunks, seq, segment;
    bool last;  // segment of its sequence
    bool odd;   // no range of the call's tokens
    int fault;
};
template <bool TRANS>
__device__ __forceinline__ Span span_of(const SsmRunArgs &p, const Segments &sg, int vs) {
    Span x;
    const int per = sg.tokens ? (TRANS ? sg.n - 1 : sg.n) : 1;
    x.seq = vs / per, x.segment = vs - x.seq * per;
    x.slot = __ldg(p.slot_ids + x.seq), x.t0 = __ldg(p.cu_seqlens + x.seq), x.t1 = __ldg(p.cu_seqlens + x.seq + 1);
    x.chunks = 0, x.last = true, x.fault = 0;
    x.odd = x.t0 < 0 || x.t1 < x.t0 || x.t1 > p.total_tokens;
    if (x.slot < 0 || x.slot >= p.lv.n_slots) {
        x.fault = WKV7_DEV_BAD_SLOT;
    } else if (x.odd || x.t1 - x.t0 > p.max_seqlen) {
        x.fault = WKV7_DEV_BAD_SEQLENS;
    } else {
        if (sg.tokens) {
            const int end = x.t1;
            if (x.segment > 0 && x.t1 - x.t0 <= static_cast<long long>(x.segment) * sg.tokens) return x;
            x.t0 += x.segment * sg.tokens;
            x.t1 = x.t0 + min(x.t1 - x.t0, sg.tokens);  // (t0 + tokens may pass 32 bits)
            x.last = x.t1 == end;
            if (TRANS && x.last) return x;
        }
        x.chunks = (x.t1 - x.t0 + kL - 1) / kL;
    }
    return x;
}

template <int NS, bool OF32, bool TRANS, bool W3>
__global__ void __launch_bounds__(kThreads, 1)
    ssm_chunk_kernel(const __grid_constant__ SsmRunArgs p, const Segments sg, const Shares sh, const __grid_constant__ Maps maps) {
    using M = Smem<NS, W3>;
    constexpr int kStagesX = M::kStagesX;
    constexpr int kStateWarps = 2 * (NS / 32);  // with something to do
    extern __shared__ uint8_t smem_raw[];
    pdl_prologue();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int halves = p.lv.p >> 6, units = p.lv.heads * halves;
    const int n_vs = p.n * (sg.tokens ? (TRANS ? sg.n - 1 : sg.n) : 1);

    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(base);
    volatile int *flag = reinterpret_cast<volatile int *>(base + M::oHold + 4);
    volatile int *redo = reinterpret_cast<volatile int *>(base + M::oHold + 8);   // some row is marked
    // (states) how a task begins for all of them: 1, there is none, 2, a wait gave up (by turns, so that none
    // is written again before all have read it); the same after the wait for another CTA
    volatile int *stop = reinterpret_cast<volatile int *>(base + M::oHold + 12);
    uint8_t *const marked = base + M::oRedo;
    Task *const tasks = reinterpret_cast<Task *>(base + M::oTask);
    uint32_t nbar = sbase + M::oBar;
    auto bars = [&nbar](int n) { const uint32_t b = nbar; nbar += 8 * n; return b; };
    const uint32_t full_c = bars(kStages), full_x = bars(kStagesX), empty_c = bars(kStages), empty_x = bars(kStagesX);
    const uint32_t full_b = bars(1), scal_ready = bars(kScal), scal_free = bars(kScal), task_ready = bars(kTasks), task_free = bars(kTasks);
    const uint32_t bar_cb = bars(1), bar_m = bars(1), bar_w = bars(1), bar_u = bars(1), u_read = bars(1), bar_s = bars(1);
    const uint32_t bar_cs = bars(1), bar_y = bars(1), y_read = bars(1), drain = bars(1);
    const long long limit = p.wait_cycles;

    // This CTA's stretch of the line of all chunks, from `spots[0]` to `spots[1]`: each thread adds up a run of
    // sequences, and finds the borders that fall into it.
    Spot *const spots = reinterpret_cast<Spot *>(base);
    int *const share = reinterpret_cast<int *>(base + 64);
    long long *const part = reinterpret_cast<long long *>(base + 128);
    if (tid == 0) *share = sh.carry ? static_cast<int>(atomicAdd(sh.drawn, 1u)) : static_cast<int>(blockIdx.x);
    if (tid < 2) spots[tid] = Spot{n_vs, 0, 0};
    const int per_thread = (n_vs + kThreads - 1) / kThreads;
    const int vs0 = static_cast<int>(min(static_cast<long long>(tid) * per_thread, static_cast<long long>(n_vs)));
    const int vs1 = static_cast<int>(min(static_cast<long long>(vs0) + per_thread, static_cast<long long>(n_vs)));
    bool none = false;  // nothing is to be run
    auto cost = [&](int vs) {
        const Span x = span_of<TRANS>(p, sg, vs);
        none |= x.odd;
        if (x.fault && blockIdx.x == 0) flag_status(p.lv.status, x.fault);
        return x.chunks ? x.chunks + kUnitCost : 0;
    };
    long long sum = 0;
    for (int vs = vs0; vs < vs1; ++vs) sum += cost(vs);
    long long upto = sum;
#pragma unroll
    for (int off = 1; off < 32; off *= 2) {
        const long long x = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += x;
    }
    if (lane == 31) part[warp] = upto;
    if (__syncthreads_or(none && p.all_or_none)) {
        if (tid == 0 && blockIdx.x == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SEQLENS);
        return;
    }
    long long before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += part[w];
        all += part[w];
    }
    upto += before;
    const int cta = *share;
    all *= units;
    // (Stretches of less than two chunks' cost could be empty, and hand nothing on.)
    const bool cut = sh.carry && all >= 2LL * gridDim.x;
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const long long at = all / gridDim.x * (cta + k) + all % gridDim.x * (cta + k) / gridDim.x;
        long long first = (upto - sum) * units;
        if (at < first || at >= upto * units) continue;
        for (int vs = vs0; vs < vs1; ++vs) {
            const long long w = cost(vs);
            if (at >= first + w * units) {
                first += w * units;
                continue;
            }
            Spot to{vs, static_cast<int>((at - first) / w), max(0, static_cast<int>((at - first) % w) - kUnitCost)};
            if (!cut) {  // units stay whole: with the CTA in whose stretch they begin
                to.unit += (at - first) % w > 0;
                to.chunk = 0;
                if (to.unit == units) {
                    to.unit = 0;
                    do ++to.vs;
                    while (to.vs < n_vs && span_of<TRANS>(p, sg, to.vs).chunks == 0);
                }
            }
            spots[k] = to;
            break;
        }
    }
    __syncthreads();
    const Spot start = spots[0], end = spots[1];
    if (start.vs == end.vs && start.unit == end.unit && start.chunk == end.chunk) return;
    __syncthreads();  // (read, before anything else is put there)

    if (warp == 0) tmem_alloc(sbase + M::oHold, 512);
    if (tid == 32) {
        for (int i = 0; i < kStages; ++i) mbar_init(full_c + 8 * i, 1), mbar_init(empty_c + 8 * i, 1);
        for (int i = 0; i < kStagesX; ++i) mbar_init(full_x + 8 * i, 1), mbar_init(empty_x + 8 * i, 4);
        mbar_init(full_b, 1);
        for (int i = 0; i < kScal; ++i)
            mbar_init(scal_ready + 8 * i, 1), mbar_init(scal_free + 8 * i, kStateWarps + (TRANS ? 0 : 4));
        for (int i = 0; i < kTasks; ++i)  // (read by states, steps, issue, scalars, and scores and outputs)
            mbar_init(task_ready + 8 * i, 1), mbar_init(task_free + 8 * i, kStateWarps + 4 + 1 + kScalWarps + (TRANS ? 0 : 12));
        mbar_init(bar_cb, 1), mbar_init(bar_m, 8), mbar_init(bar_w, 4), mbar_init(bar_u, 1), mbar_init(u_read, kStateWarps);
        mbar_init(bar_s, kStateWarps), mbar_init(bar_cs, 1), mbar_init(bar_y, 1), mbar_init(y_read, 4), mbar_init(drain, 1);
        fence_mbar_init();
        *flag = 0, *redo = 0;
    }
    if (tid < 64) marked[tid] = 0;
    if (tid < kScal) reinterpret_cast<Scal *>(base + M::oScal)[tid].after[kL - 1] = 0.f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(base + M::oHold);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    auto scal = [base](int c) { return reinterpret_cast<Scal *>(base + M::oScal + (c % kScal) * sizeof(Scal)); };
    auto wait_scal = [&](int c) { wait(scal_ready + 8 * (c % kScal), (c / kScal) & 1, flag, limit); };
    // (states) a thread's column of S, and the first of its 32 rows
    const int s_col = 32 * (warp & 3) + lane, s_row = 32 * (warp - kStateWarp >> 2);
    // Task i, which every role takes from the loads' warp, and the end of a role's use of it.  No chunks: no more.
    auto task = [&](int i) -> const Task & {
        wait(task_ready + 8 * (i % kTasks), (i / kTasks) & 1, flag, limit);
        return tasks[i % kTasks];
    };
    auto task_done = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(task_free + 8 * (i % kTasks));
    };
    // Whether a role goes on with a task, the same for the whole warp.
    auto goes_on = [&](const Task &t) { return !__any_sync(0xffffffffu, *flag != 0 || t.chunks == 0); };

    // (c counts a CTA's chunks, over all its tasks.  After a wait gave up no wait holds a role any more; the
    // roles run on to their task's end on whatever they find, all of it within bounds, and store no state of it.)
    if (warp < kStateWarp) {
        // ----------------------------------------------------------- scores
        if (!TRANS) {
            const int q = warp & 3, part = warp >> 2, t = 32 * q + lane;
            const uint32_t row = lane_base + kColM;
            float *const v = reinterpret_cast<float *>(base + M::oV) + 64 * warp;
            const int j0 = part * q, j1 = j0 + q;  // of the 2 q sets of 16 columns below the diagonal block, this warp's
            for (int i = 0, c = 0;; ++i) {
                const Task &at_task = task(i);
                if (!goes_on(at_task)) break;
#pragma unroll 1
                for (const int c1 = c + at_task.chunks; c < c1; ++c) {
                    wait_scal(c);
                    const Scal *sc = scal(c);
                    const long long gt = sc->g[t];
                    float u = 0.f;
                    if (j1 > j0) {
                        const long long border = sc->g[32 * q - 1];
                        u = ex2_fixed(gt - border);
                        __syncwarp();  // the last chunk's factors are read
                        for (int e = lane; e < 16 * (j1 - j0); e += 32) {
                            const int at = 16 * j0 + e;
                            v[e] = sc->dt[at] * ex2_fixed(border - sc->g[at]);
                        }
                        __syncwarp();
                    }
                    const F2 u2 = f2(u, u);
                    // from the diagonal's second half on its first half's decays go on from the border between them
                    float run = 0.f;
                    if (part == 0 && lane >= 16) run = ex2_fixed(gt - sc->g[32 * q + 16]);
                    wait(bar_cb, c & 1, flag, limit);
                    tc_fence_after();
                    {
                        const int k0 = 16 * part;
                        const uint32_t to = row + 32 * q + k0;
                        float x[16];
                        tmem_ld16(to, x);
                        ld_wait_for(x);
#pragma unroll 1
                        for (int k = 12; k >= 0; k -= 4) {  // columns k0 + k + 3 .. k0 + k
                            const int at = 32 * q + k0 + k, me = lane - k0 - k;
                            const float4 fd = *reinterpret_cast<const float4 *>(sc->dt + at);
                            const float4 fa = *reinterpret_cast<const float4 *>(sc->after + at);
                            float r[4];
                            r[3] = run = me == 3 ? 1.f : run * fa.w;
                            r[2] = run = me == 2 ? 1.f : run * fa.z;
                            r[1] = run = me == 1 ? 1.f : run * fa.y;
                            r[0] = run = me == 0 ? 1.f : run * fa.x;
                            uint32_t hi[2], lo[2];
                            split2(f2(x[12], x[13]) * (f2(r[0], r[1]) * f2(fd.x, fd.y)), hi[0], lo[0]);
                            split2(f2(x[14], x[15]) * (f2(r[2], r[3]) * f2(fd.z, fd.w)), hi[1], lo[1]);
                            tmem_st2(to + k / 2, hi);
                            tmem_st2(to + 8 + k / 2, lo);
#pragma unroll
                            for (int e = 15; e >= 4; --e) x[e] = x[e - 4];
                        }
                    }
#pragma unroll 1
                    for (int j = 2 * q + 2 + part; j < 8; j += 2) {
                        const uint32_t none[4] = {};
#pragma unroll
                        for (int e = 0; e < 16; e += 4) tmem_st4(row + 16 * j + e, none);
                    }
#pragma unroll 1
                    for (int j = j0; j < j1; ++j) {
                        float x[16];
                        tmem_ld16(row + 16 * j, x);
                        ld_wait_for(x);
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 f = *reinterpret_cast<const float4 *>(v + 16 * (j - j0) + 4 * e);
                            split2(f2(x[4 * e], x[4 * e + 1]) * u2 * f2(f.x, f.y), w[2 * e], w[8 + 2 * e]);
                            split2(f2(x[4 * e + 2], x[4 * e + 3]) * u2 * f2(f.z, f.w), w[2 * e + 1], w[8 + 2 * e + 1]);
                        }
                        tmem_st16(row + 16 * j, w);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_m);
                }
                task_done(i);
            }
        }
    } else if (warp < kStepWarp) {
        // ----------------------------------------------------------- states
        if (s_col < NS) {
            const uint32_t own = lane_base + kColS + s_row, add = lane_base + kColU + s_row;
            uint8_t *const to_hi = base + M::oS;
            auto hand_on = [&](int r, const F2 (&v)[4]) {  // rows s_row + r .. + 7 for C S0^T
                uint4 hi, lo;
                split2(v[0], hi.x, lo.x);
                split2(v[1], hi.y, lo.y);
                split2(v[2], hi.z, lo.z);
                split2(v[3], hi.w, lo.w);
                const uint32_t at = sw128_off(s_col, s_row + r);
                *reinterpret_cast<uint4 *>(to_hi + at) = hi;
                *reinterpret_cast<uint4 *>(to_hi + M::kS + at) = lo;
            };
            auto handed_on = [&] {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_s);
            };
            constexpr uint32_t kThreadsS = 32 * kStateWarps;
            const bool leads = warp == kStateWarp && lane == 0;
            auto load_half = [&](const Task &t, int r0, float (&v)[16]) {
                const int at = (s_row + r0) * NS + s_col;
                // (a loop for each kind: all loads on their way before the first is used)
                if (!t.from) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) v[r] = 0.f;
                } else if (t.from_bf16) {
                    const uint16_t *f = static_cast<const uint16_t *>(t.from) + at;
#pragma unroll
                    for (int r = 0; r < 16; ++r) v[r] = __uint_as_float(static_cast<uint32_t>(f[r * NS]) << 16);
                } else {
                    const float *f = static_cast<const float *>(t.from) + at;
#pragma unroll
                    for (int r = 0; r < 16; ++r) v[r] = __ldcg(f + r * NS);
                }
            };
            // From unit to unit: the last one's state is stored, the next one's taken.
            float all_decay = 1.f;
            for (int i = 0, c = 0;; ++i) {
                const Task &t = task(i);
                if (leads) stop[i & 1] = *flag ? 2 : t.chunks == 0;
                bar_sync_named(1, kThreadsS);  // all go on or none; the last unit's marks are set
                const int how = stop[i & 1];
                if (how == 2) break;
                const bool again = *redo != 0;
                if (i > 0) {  // the last unit's state goes where it belongs, but for rows that are not finite
                    const Task &old = tasks[(i - 1) % kTasks];
#pragma unroll 1
                    for (int r = 0; r < 32 && old.to; r += 8) {
                        const int at = (s_row + r) * NS + s_col;
                        float x[8];
                        tmem_ld8(own + r, x);
                        ld_wait_for(x);
                        if (again) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (!marked[s_row + r + e]) store_out(old.to, old.to_bf16, at + e * NS, x[e]);
                        } else if (old.to_bf16) {
                            __nv_bfloat16 *f = static_cast<__nv_bfloat16 *>(old.to) + at;
#pragma unroll
                            for (int e = 0; e < 8; ++e) f[e * NS] = __float2bfloat16_rn(x[e]);
                        } else {
                            float *f = static_cast<float *>(old.to) + at;
#pragma unroll
                            for (int e = 0; e < 8; ++e) f[e * NS] = x[e];
                        }
                    }
                    if (again) {
                        if (!TRANS) wait(empty_x + 8 * ((c - 1) % kStagesX), ((c - 1) / kStagesX) & 1, flag, limit);  // its outputs are out
#pragma unroll 1
                        for (int r = 4 * ((warp & 3) + (warp - kStateWarp >> 2) * (NS / 32)); r < 64; r += 4 * kStateWarps) {
                            const uint32_t mine = marked[r] | marked[r + 1] << 1 | marked[r + 2] << 2 | marked[r + 3] << 3;
                            if (mine) run_by_token<NS>(p, old, r, mine, !TRANS);
                        }
                    }
                    // No warp marks rows of the next unit before all have seen whether this one has any, nor before
                    // these are cleared.  (A unit of one chunk has nothing else that a warp waits for.)
                    if (old.signal >= 0) __threadfence();
                    bar_sync_named(1, kThreadsS);
                    if (leads && old.signal >= 0)
                        asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(sh.done + old.signal), "r"(1u) : "memory");
                    if (again) {
                        if (tid < 32 * kStateWarp + 64 && tid >= 32 * kStateWarp) marked[tid - 32 * kStateWarp] = 0;
                        if (leads) *redo = 0;
                        bar_sync_named(1, kThreadsS);
                    }
                    if (TRANS && leads) sg.decay[old.mark] = all_decay, sg.done[old.mark] = 1;
                    task_done(i - 1);
                }
                if (how) break;
                if (t.after >= 0) {  // the CTA that has this unit's first part began with it
                    if (leads) {
                        const long long since = clock64();
                        unsigned there;
                        do {
                            asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(there) : "l"(sh.done + t.after) : "memory");
                            if (!there) __nanosleep(200);
                        } while (!there && clock64() - since <= limit);
                        if (!there) *flag = 1;
                        stop[2] = *flag;
                    }
                    bar_sync_named(1, kThreadsS);
                    if (stop[2]) break;
                }
                const int chunks = t.chunks;
                if (!TRANS && c > 0) wait(bar_cs, (c - 1) & 1, flag, limit);
#pragma unroll 1
                for (int r0 = 0; r0 < 32; r0 += 16) {
                    float v[16];
                    load_half(t, r0, v);
#pragma unroll
                    for (int r = 0; r < 16; r += 8) {
                        const float x[8] = {v[r], v[r + 1], v[r + 2], v[r + 3], v[r + 4], v[r + 5], v[r + 6], v[r + 7]};
                        tmem_st8f(own + r0 + r, x);
                        const F2 w[4] = {f2(x[0], x[1]), f2(x[2], x[3]), f2(x[4], x[5]), f2(x[6], x[7])};
                        if (!TRANS) hand_on(r0 + r, w);
                    }
                }
                tmem_st_wait();
                if (!TRANS) handed_on();
                all_decay = 1.f;
#pragma unroll 1
                for (int k = 0; k < chunks; ++k, ++c) {
                    const bool more = !TRANS && k + 1 < chunks, last = k + 1 == chunks;
                    wait_scal(c);
                    const float decay = scal(c)->decay;
                    const F2 d2 = f2(decay, decay);
                    if (TRANS) all_decay *= decay;
                    wait(bar_u, c & 1, flag, limit);
                    if (more) wait(bar_cs, c & 1, flag, limit);  // the product with this chunk's S0 has read it
                    tc_fence_after();
#pragma unroll 1
                    for (int r = 0; r < 32; r += 8) {
                        float x[8], a[8], b[8];
                        tmem_ld8(own + r, x);
                        tmem_ld8(add + r, a);
                        tmem_ld8(add + 64 + r, b);
                        ld_wait_for(x);
                        ld_wait_for(a);
                        ld_wait_for(b);
                        F2 w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            w[e] = fma2(f2(x[2 * e], x[2 * e + 1]), d2, f2(a[2 * e], a[2 * e + 1]) + f2(b[2 * e], b[2 * e + 1]));
                            unpack(w[e], x[2 * e], x[2 * e + 1]);
                        }
                        tmem_st8f(own + r, x);
                        if (more) hand_on(r, w);
                        if (last) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (!finite(x[e])) marked[s_row + r + e] = 1, *redo = 1;
                        }
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    if (more) handed_on();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(u_read), mbar_arrive(scal_free + 8 * (c % kScal));
                }
            }
        }
    } else if (warp < kOutWarp) {
        // ------------------------------------------------------------ steps
        const int row = tid - 32 * kStepWarp;
        for (int i = 0, c = 0;; ++i) {
            const Task &t = task(i);
            if (!goes_on(t)) break;
            const int len = t.len;
#pragma unroll 1
            for (int k0 = 0; k0 < len; k0 += kL, ++c) {
                const int n = min(kL, len - k0);
                wait_scal(c);
                const Scal *sc = scal(c);
                const bool live = row < n;
                const float w = live ? sc->dt[row] * ex2_fixed(sc->g[kL - 1] - sc->g[row]) : 0.f;
                const F2 w2 = f2(w, w);
                wait(full_x + 8 * (c % kStagesX), (c / kStagesX) & 1, flag, limit);
                if (c > 0) wait(bar_u, (c - 1) & 1, flag, limit);
                uint8_t *const x = base + M::oX + (c % kStagesX) * kTile;
                uint8_t *const to_hi = base + M::oW;
#pragma unroll 2
                for (int i = 0; i < 8; ++i) {
                    const uint32_t at = sw128_off(row, 8 * i);
                    uint4 v = *reinterpret_cast<const uint4 *>(x + at);
                    if (!live) v = make_uint4(0, 0, 0, 0);
                    uint4 hi, lo;
                    if constexpr (W3) {
                        uint4 least;
                        split3(pair_of(v.x) * w2, hi.x, lo.x, least.x);
                        split3(pair_of(v.y) * w2, hi.y, lo.y, least.y);
                        split3(pair_of(v.z) * w2, hi.z, lo.z, least.z);
                        split3(pair_of(v.w) * w2, hi.w, lo.w, least.w);
                        *reinterpret_cast<uint4 *>(to_hi + 2 * kTile + at) = least;
                    } else {
                        split2(pair_of(v.x) * w2, hi.x, lo.x);
                        split2(pair_of(v.y) * w2, hi.y, lo.y);
                        split2(pair_of(v.z) * w2, hi.z, lo.z);
                        split2(pair_of(v.w) * w2, hi.w, lo.w);
                    }
                    *reinterpret_cast<uint4 *>(to_hi + at) = hi;
                    *reinterpret_cast<uint4 *>(to_hi + kTile + at) = lo;
                }
                if (n < kL) {  // what follows the sequence's end is zero in the products over tokens
                    wait(full_b, c & 1, flag, limit);
                    if (!live) {
#pragma unroll 1
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t at = sw128_off(row, 8 * i);
                            *reinterpret_cast<uint4 *>(x + at) = make_uint4(0, 0, 0, 0);
#pragma unroll
                            for (int k = 0; k < NS / 64; ++k)
                                *reinterpret_cast<uint4 *>(base + M::oB + k * kTile + at) = make_uint4(0, 0, 0, 0);
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar_w);
                    if (TRANS) mbar_arrive(empty_x + 8 * (c % kStagesX));
                }
            }
            task_done(i);
        }
    } else if (warp < kIssueWarp) {
        // ---------------------------------------------------------- outputs
        if (!TRANS) {
            const int q = warp - kOutWarp, t = 32 * q + lane;
            constexpr int kPasses = OF32 ? 2 : 1, kPieces = 8 / kPasses;
            for (int i = 0, c = 0;; ++i) {
                const Task &tk = task(i);
                if (!goes_on(tk)) break;
                const int len = tk.len;
                const size_t o_base = (static_cast<size_t>(tk.t0) * p.lv.heads + tk.h) * p.lv.p + tk.row0;
                const float d = p.in.d ? __ldg(p.in.d + tk.h) : 0.f;
                const F2 d2 = f2(d, d);
#pragma unroll 1
                for (int k0 = 0; k0 < len; k0 += kL, ++c) {
                    const int n = min(kL, len - k0);
                    wait_scal(c);
                    const float e = ex2_fixed(scal(c)->g[t]);
                    const F2 e2 = f2(e, e);
                    wait(bar_y, c & 1, flag, limit);
                    tc_fence_after();
                    // x's row t (it has come: the product that this waited for read it) gives way to the outputs, in
                    // two passes of float32 from its end on: what the second one needs of it is kept.
                    uint8_t *const tile = base + M::oX + (c % kStagesX) * kTile;
                    uint4 kept[4];
                    if (OF32) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) kept[k] = *reinterpret_cast<const uint4 *>(tile + sw128_off(t, 8 * (4 + k)));
                    }
#pragma unroll 1
                    for (int pass = 0; pass < kPasses; ++pass) {
#pragma unroll (OF32 ? kPieces : 1)
                        for (int i = kPieces - 1; i >= 0; --i) {
                            const uint32_t col = 8 * (pass * kPieces + i);
                            const uint4 x = pass ? kept[i & 3] : *reinterpret_cast<const uint4 *>(tile + sw128_off(t, 8 * i));
                            float y[8], a[8], b[8];
                            tmem_ld8(lane_base + kColY + col, y);
                            tmem_ld8(lane_base + kColCS + col, a);
                            tmem_ld8(lane_base + kColCS + 64 + col, b);
                            ld_wait_for(y);
                            ld_wait_for(a);
                            ld_wait_for(b);
                            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                unpack(fma2(d2, pair_of(xs[k]),
                                            fma2(e2, f2(a[2 * k], a[2 * k + 1]) + f2(b[2 * k], b[2 * k + 1]), f2(y[2 * k], y[2 * k + 1]))),
                                       y[2 * k], y[2 * k + 1]);
                            if (OF32) {
#pragma unroll
                                for (int k = 0; k < 2; ++k)
                                    *reinterpret_cast<float4 *>(tile + sw128_off(t, 8 * (2 * i + k))) =
                                        make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
                            } else {
                                *reinterpret_cast<uint4 *>(tile + sw128_off(t, 8 * i)) =
                                    make_uint4(pack_bf16_rn(y[0], y[1]), pack_bf16_rn(y[2], y[3]), pack_bf16_rn(y[4], y[5]),
                                               pack_bf16_rn(y[6], y[7]));
                            }
                        }
                        if (pass == kPasses - 1) tc_fence_before();
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (pass == kPasses - 1 && lane == 0) mbar_arrive(y_read), mbar_arrive(scal_free + 8 * (c % kScal));
                        if (32 * q + 32 <= n) {  // a warp's 32 rows of 128 bytes, as they lie
                            if (lane == 0) {
                                tma_store_3d(&maps.o, smem_addr(tile) + 4096 * q, tk.row0 + 32 * pass, tk.h, tk.t0 + k0 + 32 * q);
                                tma_store_wait<true>();
                            }
                        } else if (32 * q < n) {  // four rows at a time, up to the sequence's end
#pragma unroll 1
                            for (int r = 32 * q + (lane >> 3); r < n && r < 32 * q + 32; r += 4) {
                                const int part = lane & 7;
                                const uint4 v = *reinterpret_cast<const uint4 *>(tile + sw128_off(r, 8 * part));
                                const size_t at = o_base + static_cast<size_t>(k0 + r) * p.lv.heads * p.lv.p;
                                if (OF32) *reinterpret_cast<uint4 *>(static_cast<float *>(p.in.o) + at + 32 * pass + 4 * part) = v;
                                else *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.in.o) + at + 8 * part) = v;
                            }
                            fence_proxy_async_smem();
                        }
                        __syncwarp();
                    }
                    if (lane == 0) {
                        // The unit's rows may be run again by token: then this warp's boxes of all its chunks have to be
                        // out, also where the last chunk ends before its rows.
                        if (k0 + kL >= len) tma_store_wait<false>();
                        mbar_arrive(empty_x + 8 * (c % kStagesX));
                    }
                }
                task_done(i);
            }
        }
    } else if (warp == kIssueWarp) {
        // ------------------------------------------------------------ issue
        const uint64_t b_k = desc_sw128(sbase + M::oB), b_mn = desc_sw128_mn(sbase + M::oB, kTile);
        const uint64_t w_mn = desc_sw128_mn(sbase + M::oW, kTile), s_mn = desc_sw128_mn(sbase + M::oS, M::kS);
        const uint64_t c_k = desc_sw128(sbase + M::oC), x_mn = desc_sw128_mn(sbase + M::oX, 8192);
        for (int i = 0, c = 0;; ++i) {
            const Task &t = task(i);
            if (!goes_on(t)) break;
            const int len = t.len;
#pragma unroll 1
            for (int k0 = 0; k0 < len; k0 += kL, ++c) {
                if (__any_sync(0xffffffffu, *flag != 0)) break;
                const uint64_t c_st = c_k + (c % kStages) * (M::kState >> 4), x_st = x_mn + (c % kStagesX) * (kTile >> 4);
                wait(full_b, c & 1, flag, limit);
                if (!TRANS) {
                    wait(full_c + 8 * (c % kStages), (c / kStages) & 1, flag, limit);
                    if (len - k0 < kL) wait(bar_w, c & 1, flag, limit);  // B's rows behind the end are zeros now
                    if (c > 0) wait(bar_y, (c - 1) & 1, flag, limit);        // M X has read M
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < NS / 64; ++k)
                            umma_slices<4>(tmem + kColM, c_st + k * (kTile >> 4), 32, b_k + k * (kTile >> 4), 32, idesc_bf16_f32(128, 128), k > 0);
                        umma_commit(bar_cb);
                    }
                    __syncwarp();
                }
                wait(bar_w, c & 1, flag, limit);
                if (c > 0) wait(u_read, (c - 1) & 1, flag, limit);
                tc_fence_after();
                if (elect_one()) {
                    // (d_state 64: the second 64 rows of U are of whatever lies there, and are not read)
                    if constexpr (W3) {  // (products of one shape into the same columns run in order)
                        constexpr uint32_t idesc = idesc_bf16_f32(128, 64, 1) | (1u << 15);
#pragma unroll 1
                        for (int part = 0; part < 3; ++part)
                            umma_slices<8>(tmem + kColU + (part ? 64 : 0), b_mn, 2048, w_mn + part * (kTile >> 4), 2048, idesc, part == 2);
                    } else {
                        umma_slices<8>(tmem + kColU, b_mn, 2048, w_mn, 2048, idesc_bf16_f32(128, 128, 1) | (1u << 15), false);
                    }
                    umma_commit(bar_u);
                }
                __syncwarp();
                if (!TRANS) {
                    wait(bar_s, c & 1, flag, limit);
                    if (c > 0) wait(y_read, (c - 1) & 1, flag, limit);
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < NS / 64; ++k)
                            umma_slices<4>(tmem + kColCS, c_st + k * (kTile >> 4), 32, s_mn + k * (8192 >> 4), 2048,
                                           idesc_bf16_f32(128, 128, 1), k > 0);
                        umma_commit(bar_cs);
                        umma_commit(empty_c + 8 * (c % kStages));
                    }
                    __syncwarp();
                    wait(full_x + 8 * (c % kStagesX), (c / kStagesX) & 1, flag, limit);
                    wait(bar_m, c & 1, flag, limit);
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kL / 16; ++k) {
                            const uint32_t m = tmem + kColM + 16 * k;
                            umma_bf16_ta(tmem + kColY, m, x_st + k * (2048 >> 4), idesc_bf16_f32(128, 64, 1), k > 0 ? 1u : 0u);
                            umma_bf16_ta(tmem + kColY, m + 8, x_st + k * (2048 >> 4), idesc_bf16_f32(128, 64, 1), 1u);
                        }
                        umma_commit(bar_y);
                    }
                    __syncwarp();
                }
            }
            task_done(i);
        }
        if (elect_one()) umma_commit(drain);
        __syncwarp();
        if (lane == 0) mbar_wait_bounded(drain, 0, limit);
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            prefetch_tensormap(&maps.x);
            prefetch_tensormap(&maps.b);
            if (!TRANS) prefetch_tensormap(&maps.c);
            const bool skip = p.test_skip_loads == 1 || (TRANS && p.test_skip_loads == 2);
            int in_x = 0, in_b = 0;  // loads issued
            // first the unit that the end cuts, then the whole ones, then the rest of the one that the start cuts
            const bool rest = start.chunk > 0, one = rest && start.vs == end.vs && start.unit == end.unit;
            int stage = end.chunk > 0 && !one ? 0 : 1;
            Spot at = start;
            int known = -1;  // the sequence in x
            Span x{};
            auto step = [&] {  // to the next unit, or to the end
                if (++at.unit < units) return;
                at.unit = 0;
                do ++at.vs;
                while (at.vs < end.vs && span_of<TRANS>(p, sg, at.vs).chunks == 0);
            };
            if (rest) step();
            int sent = 0;
            auto send = [&](Task &t) {  // works out the next unit and hands it to the other roles; whether there is one
                if (sent >= kTasks) wait(task_free + 8 * (sent % kTasks), ((sent / kTasks) - 1) & 1, flag, limit);
                if (*flag) return false;
                t = Task{};
                t.after = t.signal = -1;
                Spot u = end;
                int c0 = 0, c1 = end.chunk;  // the unit's chunks
                bool found = stage == 0, to_end = false;
                if (stage == 0) {
                    stage = 1;
                } else if (stage == 1 && !one && (at.vs < end.vs || (at.vs == end.vs && at.unit < end.unit))) {
                    u = at, found = to_end = true;
                    step();
                } else if (rest && stage < 2) {
                    stage = 2;
                    u = start, c0 = start.chunk, found = true, to_end = !one;
                    t.after = cta - 1;
                }
                if (found) {
                    if (u.vs != known) x = span_of<TRANS>(p, sg, u.vs), known = u.vs;
                    if (to_end) c1 = x.chunks;
                    else t.signal = cta;
                    t.h = u.unit / halves, t.row0 = (u.unit - t.h * halves) * 64;
                    t.chunks = c1 - c0;
                    t.t0 = x.t0 + c0 * kL;
                    t.len = min(x.t1, x.t0 + c1 * kL) - t.t0;
                    const size_t esz = p.lv.state_bf16 ? 2 : 4;
                    char *const own = reinterpret_cast<char *>(p.lv.states) +
                                      (static_cast<size_t>(x.slot) * p.lv.slot_stride + p.lv.layer_off +
                                       (static_cast<size_t>(t.h) * p.lv.p + t.row0) * NS) * esz;
                    const size_t unit = static_cast<size_t>(x.seq) * units + u.unit;
                    t.from = own, t.to = own, t.from_bf16 = t.to_bf16 = p.lv.state_bf16;
                    int lost = 0;
                    if (TRANS) {
                        t.from = nullptr, t.from_bf16 = 0;
                        t.to = sg.state + (unit * sg.n + x.segment + 1) * (64 * NS), t.to_bf16 = 0;
                        t.mark = static_cast<long long>(unit) * (sg.n - 1) + x.segment;
                    } else if (sg.tokens && (x.segment > 0 || !x.last)) {
                        t.from = sg.state + (unit * sg.n + x.segment) * (64 * NS), t.from_bf16 = 0;
                        if (!x.last) t.to = nullptr;
                        lost = sg.lost[unit];
                    }
                    if (t.after >= 0) t.from = sh.carry + static_cast<size_t>(t.after) * (64 * NS), t.from_bf16 = 0;
                    if (t.signal >= 0) t.to = sh.carry + static_cast<size_t>(cta) * (64 * NS), t.to_bf16 = 0;
                    if (lost) *flag = 1;  // what it starts from was never written
                }
                tasks[sent % kTasks] = t;
                mbar_arrive(task_ready + 8 * (sent % kTasks));
                ++sent;
                if (found && t.from && t.after < 0)  // on its way before the states' warps ask for it
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(t.from), "r"(64 * NS * (t.from_bf16 ? 2 : 4)) : "memory");
                return found;
            };
            Task t, next;
            bool more = send(t);
            for (int c = 0; more && !*flag;) {
                more = send(next);  // a unit ahead
                const int g = t.h / (p.lv.heads / p.lv.groups);
#pragma unroll 1
                for (int k = 0; k < t.chunks && !skip; ++k, ++c) {
                    const int st = c % kStages, sx = c % kStagesX, tok = t.t0 + k * kL;
                    if (!TRANS && c >= kStages) wait(empty_c + 8 * st, ((c / kStages) - 1) & 1, flag, limit);
                    if (c >= kStagesX) wait(empty_x + 8 * sx, ((c / kStagesX) - 1) & 1, flag, limit);
                    if (*flag) break;
                    if (!TRANS) {
                        mbar_arrive_expect_tx(full_c + 8 * st, M::kState);
#pragma unroll
                        for (int q = 0; q < NS / 64; ++q)
                            tma_load_3d(sbase + M::oC + st * M::kState + q * kTile, &maps.c, 64 * q, g, tok, full_c + 8 * st);
                    }
                    mbar_arrive_expect_tx(full_x + 8 * sx, kTile);
                    tma_load_3d(sbase + M::oX + sx * kTile, &maps.x, t.row0, t.h, tok, full_x + 8 * sx);
                    ++in_x;
                    if (c > 0) wait(bar_u, (c - 1) & 1, flag, limit);
                    if (*flag) break;
                    ++in_b;
                    mbar_arrive_expect_tx(full_b, M::kState);
#pragma unroll
                    for (int q = 0; q < NS / 64; ++q) tma_load_3d(sbase + M::oB + q * kTile, &maps.b, 64 * q, g, tok, full_b);
                }
                t = next;
            }
            if (*flag) {  // what is on its way must arrive before the CTA ends
                for (int k = max(0, in_x - kStages); k < in_x && !TRANS; ++k)
                    mbar_wait_bounded(full_c + 8 * (k % kStages), (k / kStages) & 1, limit);
                for (int k = max(0, in_x - kStagesX); k < in_x; ++k)
                    mbar_wait_bounded(full_x + 8 * (k % kStagesX), (k / kStagesX) & 1, limit);
                if (in_b > 0) mbar_wait_bounded(full_b, (in_b - 1) & 1, limit);
            }
        }
    } else {
        // ---------------------------------------------------------- scalars
        // A chunk in four runs of 32 tokens, a token a lane; the next chunk's dt is loaded as it comes, from
        // addresses that always exist, so that nothing waits for it before it is used.
        constexpr float kLog2e = 1.4426950408889634f;
        const int mine = warp - kScalWarp;
        const bool biased = p.in.dt_bias != nullptr;
        for (int i = 0, c0 = 0;; ++i) {
            const Task &t = task(i);
            if (!goes_on(t)) break;
            const int len = t.len, h = t.h, chunks = t.chunks;
            const long long t0 = t.t0;
            const float a2 = __ldg(p.in.a + h), bias = biased ? __ldg(p.in.dt_bias + h) : 0.f;
            auto tokens_of = [&](int k, uint32_t (&raw)[4]) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const size_t at = static_cast<size_t>((t0 + min(k * kL + 32 * e + lane, len - 1)) * p.in.dt_stride + h);
                    raw[e] = p.in.dt_bf16 ? static_cast<uint32_t>(__ldg(static_cast<const unsigned short *>(p.in.dt) + at))
                                          : __ldg(static_cast<const uint32_t *>(p.in.dt) + at);
                }
            };
            uint32_t raw[4], next[4];
            const int k0 = (mine + c0) & 1;
            tokens_of(k0, raw);
#pragma unroll 1
            for (int k = k0; k < chunks; k += kScalWarps) {
                const int c = c0 + k;
                tokens_of(k + kScalWarps, next);
                if (c >= kScal) wait(scal_free + 8 * (c % kScal), ((c / kScal) - 1) & 1, flag, limit);
                __syncwarp();
                Scal *sc = scal(c);
                long long upto = 0;  // the sum up to this run
#pragma unroll 1
                for (int e = 0; e < 4; ++e) {
                    const int at = 32 * e + lane;
                    const bool live = k * kL + at < len;
                    const float x = __uint_as_float(p.in.dt_bf16 ? raw[0] << 16 : raw[0]);
                    const float y = biased ? __fadd_rn(x, bias) : x;
                    float dt = live ? p.in.softplus ? softplus(y) : y : 0.f;
                    const float g = live ? __fmul_rn(__fmul_rn(dt, a2), kLog2e) : 0.f;
                    if (g != g) dt = g;  // a NaN reaches M and U through the step; the sum takes it for -160
                    const float bound = fminf(fmaxf(g, -160.f), 160.f);
                    long long sum = __float2ll_rn(bound * 0x1p40f);
#pragma unroll
                    for (int off = 1; off < 32; off *= 2) {
                        const long long before = __shfl_up_sync(0xffffffffu, sum, off);
                        if (lane >= off) sum += before;
                    }
                    sum += upto;
                    sc->g[at] = sum;
                    sc->dt[at] = dt;
                    if (at > 0) sc->after[at - 1] = ex2_approx(bound);
                    upto = __shfl_sync(0xffffffffu, sum, 31);
                    raw[0] = raw[1], raw[1] = raw[2], raw[2] = raw[3];
                }
                if (lane == 31) sc->decay = ex2_fixed(upto);
                __syncwarp();
                if (lane == 0) mbar_arrive(scal_ready + 8 * (c % kScal));
#pragma unroll
                for (int e = 0; e < 4; ++e) raw[e] = next[e];
            }
            c0 += chunks;
            task_done(i);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *flag) flag_status(p.lv.status, WKV7_DEV_WAIT_TIMEOUT);
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// The states at the segments' starts, S_{j+1} = d_j S_j + what segment j leaves from zero, written over that;
// at 0 a copy of the slot's state (the last segment may store its own there before the first has read it).
constexpr int kJoinThreads = 256;

template <int NS>
__global__ void __launch_bounds__(kJoinThreads) ssm_join_kernel(const SsmRunArgs p, const Segments sg) {
    pdl_prologue();
    const int seq = blockIdx.z, halves = p.lv.p >> 6, h = blockIdx.y / halves, row0 = (blockIdx.y - h * halves) * 64;
    const int slot = __ldg(p.slot_ids + seq), t0 = __ldg(p.cu_seqlens + seq), t1 = __ldg(p.cu_seqlens + seq + 1);
    if (slot < 0 || slot >= p.lv.n_slots) return;  // (flagged before)
    if (t0 < 0 || t1 < t0 || t1 > p.total_tokens || t1 - t0 > p.max_seqlen) return;
    const int n = t1 > t0 ? min(sg.n, (t1 - t0 - 1) / sg.tokens + 1) : 0;  // this sequence's segments
    if (n < 2) return;  // (it starts from its slot)
    const size_t unit = static_cast<size_t>(seq) * gridDim.y + blockIdx.y;
    int lost = 0;
    for (int j = 0; j < n - 1; ++j) lost |= !sg.done[unit * (sg.n - 1) + j];
    if (blockIdx.x == 0 && threadIdx.x == 0) sg.lost[unit] = lost;
    if (lost) return;
    const int at = (blockIdx.x * kJoinThreads + threadIdx.x) * 4;
    const size_t off = static_cast<size_t>(slot) * p.lv.slot_stride + p.lv.layer_off + (static_cast<size_t>(h) * p.lv.p + row0) * NS + at;
    float4 s = p.lv.state_bf16 ? load_state4<true>(p.lv.states, off) : load_state4<false>(p.lv.states, off);
    float4 *to = reinterpret_cast<float4 *>(sg.state + unit * sg.n * (64 * NS) + at);
    constexpr int kStep = 64 * NS / 4;
    *to = s;
    float4 next = to[kStep];
    for (int j = 1; j < n; ++j) {
        const float4 left = next;
        if (j + 1 < n) next = to[(j + 1) * kStep];
        const float d = sg.decay[unit * (sg.n - 1) + j - 1];
        s.x = fmaf(d, s.x, left.x), s.y = fmaf(d, s.y, left.y), s.z = fmaf(d, s.z, left.z), s.w = fmaf(d, s.w, left.w);
        to[j * kStep] = s;
    }
}

// ------------------------------------------------------------------ host side

// [tokens][heads][size] with rows `stride` elements apart; one box = `rows` tokens x 1 head x 128 bytes,
// swizzled as the tiles are, zeros past the end.
bool encode(CUtensorMap *map, const void *ptr, int size, int heads, int tokens, long long stride, bool f32 = false, int rows = kL) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t esz = f32 ? 4 : 2;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(size), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(size) * esz, static_cast<cuuint64_t>(stride) * esz};
    cuuint32_t box[3] = {f32 ? 32u : 64u, 1, static_cast<cuuint32_t>(rows)};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims,
               strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kSms = 152;

template <int NS, bool OF32, bool TRANS, bool W3>
cudaError_t launch_chunks_as(const SsmRunArgs &a, const Segments &sg, const Shares &sh, const Maps &maps, cudaStream_t s) {
    constexpr int bytes = static_cast<int>(Smem<NS, W3>::kBytes) + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
    auto kernel = ssm_chunk_kernel<NS, OF32, TRANS, W3>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return e != cudaSuccess ? e : launch_pdl(kernel, dim3(kSms), dim3(kThreads), bytes, s, a, sg, sh, maps);
}

template <int NS, bool OF32, bool TRANS>
cudaError_t launch_chunks(const SsmRunArgs &a, const Segments &sg, const Shares &sh, const Maps &maps, cudaStream_t s) {
    return a.lv.state_bf16 ? launch_chunks_as<NS, OF32, TRANS, true>(a, sg, sh, maps, s)
                           : launch_chunks_as<NS, OF32, TRANS, false>(a, sg, sh, maps, s);
}

__global__ void clear_words(unsigned *x, long long n) {
    pdl_prologue();
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < n) x[i] = 0;
}
template <int NS, bool OF32>
cudaError_t chunk_as(const SsmRunArgs &a, const SsmSplit &split, cudaStream_t s, int *launches) {
    Maps maps;
    if (!encode(&maps.x, a.in.x, a.lv.p, a.lv.heads, a.total_tokens, a.in.x_stride) ||
        !encode(&maps.b, a.in.b, NS, a.lv.groups, a.total_tokens, a.in.b_stride) ||
        !encode(&maps.c, a.in.c, NS, a.lv.groups, a.total_tokens, a.in.c_stride) ||
        !encode(&maps.o, a.in.o, a.lv.p, a.lv.heads, a.total_tokens, static_cast<long long>(a.lv.heads) * a.lv.p, OF32, 32))
        return cudaErrorInvalidValue;
    const unsigned n = static_cast<unsigned>(a.n), x = static_cast<unsigned>(a.lv.heads * (a.lv.p / 64));
    Segments sg{};
    Shares sh{};
    cudaError_t e = cudaSuccess;
    const size_t units = static_cast<size_t>(n) * x, state = 64 * NS;
    float *at = static_cast<float *>(a.workspace);  // (ssm_split_bytes adds up the same)
    if (split.segments >= 2) {
        sg.tokens = split.chunks * kL;
        sg.n = split.segments;
        sg.state = at, at += units * sg.n * state;
        sg.decay = at, at += units * (sg.n - 1);
        sg.lost = reinterpret_cast<int *>(at), at += units;
    }
    if (split.cut) sh.carry = at, at += kSms * state;
    unsigned *const flags = reinterpret_cast<unsigned *>(at);
    size_t n_flags = 0;
    if (split.segments >= 2) sg.done = reinterpret_cast<int *>(flags), n_flags = units * (sg.n - 1);
    if (split.cut) sh.done = flags + n_flags, sh.drawn = sh.done + kSms, n_flags += kSms + 1;
    if (n_flags) {
        ++*launches;
        e = launch_pdl(clear_words, dim3(static_cast<unsigned>((n_flags + 255) / 256)), dim3(256), 0, s, flags, static_cast<long long>(n_flags));
        if (e != cudaSuccess) return e;
    }
    if (split.segments >= 2) {
        e = launch_chunks<NS, false, true>(a, sg, Shares{}, maps, s);
        ++*launches;
        if (e != cudaSuccess) return e;
        e = launch_pdl(ssm_join_kernel<NS>, dim3(64 * NS / 4 / kJoinThreads, x, n), dim3(kJoinThreads), 0, s, a, sg);
        ++*launches;
        if (e != cudaSuccess) return e;
    }
    ++*launches;
    return launch_chunks<NS, OF32, false>(a, sg, sh, maps, s);
}

}  // namespace

bool ssm_chunk_takes(const SsmRunArgs &a) {
    return a.in.bf16 && a.cu_seqlens && a.total_tokens > 0 && a.in.x_stride > 0 && a.in.b_stride > 0 && a.in.c_stride > 0;
}

// Measured, us: a chunk 2.45, without outputs 1.2, a unit's start and end 4, a launch's 8, a join 4.  Where units fill
// the SMs, they are cut where an SM's share ends.  Else the number of segments that gives the shortest
// estimate, if that promises a fifth less than the uncut time; where these fill the SMs they are cut in turn.
SsmSplit ssm_plan_split(int n_seqs, int heads, int p, int max_seqlen) {
    SsmSplit best{};
    const long long units = static_cast<long long>(n_seqs) * heads * (p / 64);
    const int chunks = (max_seqlen + kL - 1) / kL;
    if (units >= kSms) {
        best.cut = chunks >= 4;
        return best;
    }
    if (units <= 0 || chunks < 8 || n_seqs > 65535) return best;
    constexpr double kStartUs = 8, kUnitUs = 4, kChunkUs = 2.45, kTransUs = 1.2, kJoinUs = 4;
    auto rounds = [](long long ctas) { return static_cast<double>((ctas + kSms - 1) / kSms); };
    double least = 0.8 * (kStartUs + kUnitUs + kChunkUs * chunks);
    for (int n = 2; n <= 128 && n * 2 <= chunks; ++n) {
        const int per = (chunks + n - 1) / n;
        if ((chunks + per - 1) / per != n) continue;
        const bool full = units * n >= kSms;
        const double last = full ? (kChunkUs * chunks + kUnitUs * n) * static_cast<double>(units) / kSms + kUnitUs
                                 : kChunkUs * per + kUnitUs;
        const double t = kStartUs + rounds(units * (n - 1)) * (kUnitUs + kTransUs * per) + kJoinUs + kStartUs + last;
        if (t < least) {
            least = t;
            best.segments = n;
            best.chunks = per;
            best.cut = full;
        }
    }
    return best;
}

size_t ssm_split_bytes(const SsmSplit &split, long long units, int ds) {
    const size_t n = static_cast<size_t>(split.segments), u = static_cast<size_t>(units), state = static_cast<size_t>(64) * ds;
    size_t words = 0;
    if (split.segments >= 2) words += u * (n * state + (n - 1) + 1 + (n - 1));
    if (split.cut) words += kSms * state + kSms + 1;
    return (words * 4 + 15) / 16 * 16;
}

cudaError_t launch_ssm_chunk(const SsmRunArgs &a, cudaStream_t s, int *launches) {
    SsmSplit split = ssm_plan_split(a.n, a.lv.heads, a.lv.p, a.max_seqlen);
    if (!a.workspace || a.workspace_bytes < ssm_split_bytes(split, static_cast<long long>(a.n) * a.lv.heads * (a.lv.p / 64), a.lv.ds))
        split = SsmSplit{};
    cudaError_t (*const as[4])(const SsmRunArgs &, const SsmSplit &, cudaStream_t, int *) = {chunk_as<64, false>, chunk_as<64, true>,
                                                                                             chunk_as<128, false>, chunk_as<128, true>};
    const cudaError_t e = as[(a.lv.ds == 128 ? 2 : 0) | (a.in.o_bf16 ? 0 : 1)](a, split, s, launches);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace wkv7
