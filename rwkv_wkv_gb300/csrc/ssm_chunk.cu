// The selective scan over whole sequences, by chunks of 128 tokens on the tcgen05 tensor cores.
//
// Per head, S [p][n], a token does  S <- exp(g) S + (dt x) B^T,  o = S C + D x,  g = dt A.
// Over a chunk from state S0, with G_t the sum of g up to token t, unrolling gives
//     O   = diag(exp G) C S0^T + M X,   M_ts = exp(G_t - G_s) dt_s <C_t, B_s> for s < t,
//                                       M_tt = dt_t <C_t, B_t> + D
//     S_L = exp(G_L) S0 + X^T diag(dt exp(G_L - G)) B
// All factors are exp of sums of g over s + 1 .. t, so at most 1: no decay is too strong.  G
// is kept as a pair of floats, so that a difference stays exact after a token that empties
// the state (g log2 e is taken as at least -160; 2^-160 is 0 in float32).
//
// Precision.  x, B and C are bf16 and go to the tensor cores as they were loaded.  The computed
// operands (S0, M, the weighted X) are split into two bf16 parts, 16 bits, which leave 2^-18 of them.
// Sums and states are float32; the states stay in tensor memory from chunk to chunk.
//
// One CTA owns 64 rows (of p) of one (sequence, head) and walks its chunks.  Its warps:
//   scores (0-7)    row t of M from C B^T, in tensor memory, back in its place: warps 0-3 the diagonal
//                   blocks of 32 x 32, 4-7 what lies below them
//   states (8-15)   column j of S, 32 of its 64 values a thread; two bf16 parts of it for the next chunk's C S0^T
//   steps (16-19)   row s of the weighted X
//   outputs (20-23) row t of O
//   issue (24)      the MMAs;  scalars (25, 26) G and dt of each token, every other chunk;  loads (27) TMA
// Four products a chunk, all of M = 128:
//     C B^T          N = 128 (s), K = n
//     U = B^T [Xh Xl]    N = 128, K = 128 (s); the halves add up
//     C [Sh Sl]      N = 128, K = n; the halves add up
//     [Mh Ml] X      N = 64, K = 2 x 128 (s), M from tensor memory
// Below its diagonal blocks of 32 x 32, M's decays are products of two factors at most 1 that meet at the
// border before row t's block: one 2^x a row and 32 a diagonal row, not one an entry.
//
// Values that are not finite.  In a product over the tokens of a chunk a zero coefficient does not keep a
// NaN or an infinity of a later token away from an earlier one, as the formulas do.  A row of S that
// meets one in x, B or dt has an entry that is not finite from then on, so such rows show in the
// CTA's last state: they are marked, and run through the CTA's tokens once more, one by one in float32.
//
// Few (sequence, head) units leave SMs idle, so long sequences are then cut into segments of whole chunks:
// TRANS runs each segment but the last from zero, without outputs; ssm_join_kernel chains the segments'
// states (S <- d S + that, d the segment's decay); then the ordinary kernel runs all segments side by side.
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
// Warps, each role's first (scores begin at 0).  28 leave 72 registers a thread, which every role keeps to: a
// value spilled goes through an L1 that shared memory leaves almost nothing of.
constexpr int kStateWarp = 8, kStepWarp = 16, kOutWarp = 20, kIssueWarp = 24, kScalWarp = 25, kScalWarps = 2, kLoadWarp = 27;
constexpr int kThreads = 28 * 32;
constexpr int kStages = 2, kStagesX = 3, kScal = 4;
constexpr int kMaxOrder = 512;  // sequences that are put in order

// Tensor-memory columns (512 allocated): C B^T, then M in its place (of each 16 columns, 8 of the
// high parts and 8 of the low ones, K elements 2c, 2c + 1 in a column); M X; C S0 in two halves; U in two
// halves; S, column j in lane j.
constexpr uint32_t kColM = 0, kColY = 128, kColCS = 192, kColU = 320, kColS = 448;

constexpr uint32_t kTile = 16384;  // 128 rows of 128 bytes, 128-byte swizzle

// A chunk's per-token values: G as a pair, in units of log 2, and dt; after them exp(G_L).
struct Scal {
    float gh[kL], gl[kL], dt[kL];
    float decay, pad[3];
};

template <int NS>
struct Smem {
    static constexpr uint32_t kState = NS / 64 * kTile;     // a tile of B or C
    static constexpr uint32_t oC = 0;                       // per stage
    static constexpr uint32_t oX = oC + kStages * kState;   // per stage; the outputs pass through it
    static constexpr uint32_t oB = oX + kStagesX * kTile;
    static constexpr uint32_t oW = oB + kState;             // the weighted X, high parts then low
    static constexpr uint32_t oS = oW + 2 * kTile;          // S: rows j of 64 (p), high parts then low
    static constexpr uint32_t kS = NS * 128;
    static constexpr uint32_t oScal = oS + 2 * kS;
    static constexpr uint32_t oV = oScal + kScal * sizeof(Scal);  // per scores warp q: 32 q border factors
    static constexpr uint32_t oBar = oV + 6 * 32 * 4;
    static constexpr uint32_t kBars = 2 * kStages + 2 * kStagesX + 1 + 2 * kScal + 10;
    static constexpr uint32_t oHold = oBar + kBars * 8;
    static constexpr uint32_t oRedo = oHold + 16;  // per row: marked (see the file's header)
    static constexpr uint32_t kBytes = oRedo + 64;
};

struct Maps {
    CUtensorMap x, b, c;
};

// A cut sequence's segments: `tokens` each (a multiple of 128; 0: not cut).  state[unit][n][64][NS]: what
// segment j alone leaves from zero at j + 1, after the join the state that segment j starts from at j;
// decay, gave_up [unit][n - 1], lost [unit]: whether a wait gave up, and then the unit's outcome is not stored.
struct Segments {
    int tokens, n;
    float *state, *decay;
    int *gave_up, *lost;
};

__device__ __forceinline__ F2 pair_of(uint32_t bf16x2) { return f2_bf16(bf16x2); }

__device__ __forceinline__ void two_sum(float a, float b, float &s, float &e) {
    s = __fadd_rn(a, b);
    const float bb = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}
// (h, l) += (x, y), renormalised.
__device__ __forceinline__ void pair_add(float &h, float &l, float x, float y) {
    float s, e;
    two_sum(h, x, s, e);
    e = __fadd_rn(e, __fadd_rn(l, y));
    h = __fadd_rn(s, e);
    l = __fsub_rn(e, __fsub_rn(h, s));
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
// 2^(a - b) of pairs.
__device__ __forceinline__ float ex2_diff(float ah, float al, float bh, float bl) {
    return ex2_approx(__fadd_rn(__fsub_rn(ah, bh), __fsub_rn(al, bl)));
}

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

// Tokens t0 .. t0 + len - 1 of the marked rows of 64 of one head (row0 the first), one by one in float32,
// by the first 16 warps of a CTA, four rows each.  From null: from zero.  Rare, so written to be small.
template <int NS>
__device__ __noinline__ void run_by_token(const SsmRunArgs &p, const uint8_t *marked, int h, int row0, int t0, int len,
                                          const float *from, size_t from_off, bool from_bf16, float *to, size_t to_off,
                                          bool to_bf16, bool outputs) {
    constexpr int R = 4, C = NS / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp >= 16) return;
    uint32_t mine = 0;
#pragma unroll
    for (int m = 0; m < R; ++m) mine |= static_cast<uint32_t>(marked[warp * R + m]) << m;
    if (mine == 0) return;
    const size_t at = static_cast<size_t>(warp * R) * NS + lane * C;
    float s[R][C];
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const size_t x = from_off + at + m * NS + c;
            s[m][c] = !from ? 0.f : from_bf16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(from)[x]) << 16)
                                              : from[x];
        }
    const int g = h / (p.lv.heads / p.lv.groups);
    const float d = p.in.d ? __ldg(p.in.d + h) : 0.f;
#pragma unroll 1
    for (int t = 0; t < len; ++t) {
        const long long row = static_cast<long long>(t0) + t;
        const StepScalars sc = step_scalars(p.in, h, load_dt(p.in, row, h));
        float b[C], c[C];
#pragma unroll
        for (int e = 0; e < C; ++e) {
            b[e] = load1<true>(p.in.b, row * p.in.b_stride + static_cast<long long>(g) * NS + lane * C + e);
            c[e] = load1<true>(p.in.c, row * p.in.c_stride + static_cast<long long>(g) * NS + lane * C + e);
        }
#pragma unroll
        for (int m = 0; m < R; ++m) {
            const int i = row0 + warp * R + m;
            const float x = load1<true>(p.in.x, row * p.in.x_stride + static_cast<long long>(h) * p.lv.p + i);
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
                store_out(p.in.o, p.in.o_bf16, (static_cast<size_t>(row) * p.lv.heads + h) * p.lv.p + i, p.in.d ? fmaf(d, x, y) : y);
        }
    }
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (to && (mine >> m & 1)) store_out(to, to_bf16, to_off + at + m * NS + c, s[m][c]);
}

template <int NS, bool OF32, bool TRANS>
__global__ void __launch_bounds__(kThreads, 1)
    ssm_chunk_kernel(const __grid_constant__ SsmRunArgs p, const Segments sg, const __grid_constant__ Maps maps) {
    using M = Smem<NS>;
    constexpr int kStateWarps = 2 * (NS / 32);  // with something to do
    extern __shared__ uint8_t smem_raw[];
    pdl_prologue();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int halves = p.lv.p >> 6;
    const int h = blockIdx.x / halves, row0 = (blockIdx.x - h * halves) * 64;
    int seq = blockIdx.y + (sg.tokens ? 0 : blockIdx.z * 65535);
    if (seq >= p.n) return;
    int slot, t0, t1;
    if (!sg.tokens && p.n > 1 && p.n <= kMaxOrder) {  // the longest sequences start first: their ends are not the grid's
        int *key = reinterpret_cast<int *>(smem_raw);
        int4 *found = reinterpret_cast<int4 *>(key + kMaxOrder);
        int4 mine{};  // of sequence tid
        if (tid < p.n) {
            mine = make_int4(tid, __ldg(p.slot_ids + tid), __ldg(p.cu_seqlens + tid), __ldg(p.cu_seqlens + tid + 1));
            key[tid] = (mine.w - mine.z + kL - 1) / kL;
        }
        __syncthreads();
        if (tid < p.n) {
            const int own = key[tid];
            int rank = 0;
#pragma unroll 8
            for (int r = 0; r < p.n; ++r) rank += key[r] > own || (key[r] == own && r < tid);
            if (rank == seq) *found = mine;
        }
        __syncthreads();
        seq = found->x, slot = found->y, t0 = found->z, t1 = found->w;
        __syncthreads();
    } else {
        slot = __ldg(p.slot_ids + seq), t0 = __ldg(p.cu_seqlens + seq), t1 = __ldg(p.cu_seqlens + seq + 1);
    }
    if (slot < 0 || slot >= p.lv.n_slots) {
        if (tid == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SLOT);
        return;
    }
    if (t0 < 0 || t1 < t0 || t1 > p.total_tokens || t1 - t0 > p.max_seqlen) {
        if (tid == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SEQLENS);
        return;
    }
    // this CTA's part of the sequence, and where its state comes from and goes to
    const float *from = TRANS ? nullptr : p.lv.states;  // (null: zeros)
    float *to = p.lv.states;
    bool from_bf16 = p.lv.state_bf16, to_bf16 = p.lv.state_bf16;
    int lost = 0;  // the start state: a wait gave up
    size_t from_off = static_cast<size_t>(slot) * p.lv.slot_stride + p.lv.layer_off + (static_cast<size_t>(h) * p.lv.p + row0) * NS;
    size_t to_off = from_off;
    bool store = true;
    const size_t unit = static_cast<size_t>(seq) * gridDim.x + blockIdx.x;
    const int segment = blockIdx.z;
    if (sg.tokens) {
        const int end = t1;
        if (segment > 0 && t1 - t0 <= static_cast<long long>(segment) * sg.tokens) return;
        t0 += segment * sg.tokens;
        t1 = min(t1, t0 + sg.tokens);
        if (TRANS) {
            if (t1 == end) return;
            to = sg.state;
            to_off = (unit * sg.n + segment + 1) * (64 * NS);
            to_bf16 = false;
        } else {
            store = t1 == end;
            if (segment > 0 || !store) {
                from = sg.state;
                from_bf16 = false;
                from_off = (unit * sg.n + segment) * (64 * NS);
                lost = sg.lost[unit];
            }
        }
    }
    const int len = t1 - t0;
    if (len == 0) return;
    const int n_chunks = (len + kL - 1) / kL;

    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(base);
    volatile int *flag = reinterpret_cast<volatile int *>(base + M::oHold + 4);
    volatile int *redo = reinterpret_cast<volatile int *>(base + M::oHold + 8);  // some row is marked
    uint8_t *const marked = base + M::oRedo;
    float *const total = reinterpret_cast<float *>(base + M::oV);  // (TRANS) the scalars' warps' sums, pairs
    uint32_t nbar = sbase + M::oBar;
    auto bars = [&nbar](int n) { const uint32_t b = nbar; nbar += 8 * n; return b; };
    const uint32_t full_c = bars(kStages), full_x = bars(kStagesX), empty_c = bars(kStages), empty_x = bars(kStagesX);
    const uint32_t full_b = bars(1), scal_ready = bars(kScal), scal_free = bars(kScal);
    const uint32_t bar_cb = bars(1), bar_m = bars(1), bar_w = bars(1), bar_u = bars(1), u_read = bars(1), bar_s = bars(1);
    const uint32_t bar_cs = bars(1), bar_y = bars(1), y_read = bars(1), drain = bars(1);
    const long long limit = p.wait_cycles;

    if (warp == 0) tmem_alloc(sbase + M::oHold, 512);
    if (tid == 32) {
        for (int i = 0; i < kStages; ++i) mbar_init(full_c + 8 * i, 1), mbar_init(empty_c + 8 * i, 1);
        for (int i = 0; i < kStagesX; ++i) mbar_init(full_x + 8 * i, 1), mbar_init(empty_x + 8 * i, 4);
        mbar_init(full_b, 1);
        for (int i = 0; i < kScal; ++i)
            mbar_init(scal_ready + 8 * i, 1), mbar_init(scal_free + 8 * i, kStateWarps + (TRANS ? 0 : 4));
        mbar_init(bar_cb, 1), mbar_init(bar_m, 8), mbar_init(bar_w, 4), mbar_init(bar_u, 1), mbar_init(u_read, kStateWarps);
        mbar_init(bar_s, kStateWarps), mbar_init(bar_cs, 1), mbar_init(bar_y, 1), mbar_init(y_read, 4), mbar_init(drain, 1);
        fence_mbar_init();
        *flag = lost, *redo = 0;
    }
    if (tid < 64) marked[tid] = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(base + M::oHold);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    auto scal = [base](int c) { return reinterpret_cast<Scal *>(base + M::oScal + (c % kScal) * sizeof(Scal)); };
    auto wait_scal = [&](int c) { wait(scal_ready + 8 * (c % kScal), (c / kScal) & 1, flag, limit); };
    // (states) a thread's column of S, and the first of its 32 rows
    const int s_col = 32 * (warp & 3) + lane, s_row = 8 * (warp & 4);

    // (After a wait gave up no wait holds a role any more; the roles run on to their end on whatever they
    // find, all of it within bounds, and nothing of it is stored as a state.)
    if (warp < kStateWarp) {
        // ----------------------------------------------------------- scores
        if (!TRANS) {
            const int q = warp & 3, t = 32 * q + lane;
            const uint32_t row = lane_base + kColM;
            float *const v = reinterpret_cast<float *>(base + M::oV) + 32 * (q * (q - 1) / 2);
            const float d = p.in.d ? __ldg(p.in.d + h) : 0.f;
#pragma unroll 1
            for (int c = 0; c < n_chunks; ++c) {
                wait_scal(c);
                const Scal *sc = scal(c);
                const float th = sc->gh[t], tl = sc->gl[t];
                if (warp < 4) {
                    wait(bar_cb, c & 1, flag, limit);
                    tc_fence_after();
                    const F2 less = f2(-1.f, -1.f), th2 = f2(th, th), tl2 = f2(tl, tl);
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t to = row + 32 * q + 16 * half;
                        float x[16];
                        tmem_ld16(to, x);
                        ld_wait_for(x);
#pragma unroll 1
                        for (int part = 0; part < 2; ++part) {
                            const int at = 16 * half + 8 * part;
                            uint32_t hi[4], lo[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 fh = *reinterpret_cast<const float2 *>(sc->gh + 32 * q + at + 2 * i);
                                const float2 fl = *reinterpret_cast<const float2 *>(sc->gl + 32 * q + at + 2 * i);
                                const float2 fd = *reinterpret_cast<const float2 *>(sc->dt + 32 * q + at + 2 * i);
                                float a, b;
                                unpack(fma2(f2(fh.x, fh.y), less, th2) + fma2(f2(fl.x, fl.y), less, tl2), a, b);
                                unpack(f2(x[2 * i], x[2 * i + 1]) * f2(fd.x, fd.y) * f2(ex2_approx(a), ex2_approx(b)), a, b);
                                const int k = at + 2 * i;
                                a = k < lane ? a : k == lane ? a + d : 0.f;
                                b = k + 1 < lane ? b : k + 1 == lane ? b + d : 0.f;
                                split2(f2(a, b), hi[i], lo[i]);
                            }
                            tmem_st4(to + 4 * part, hi);
                            tmem_st4(to + 8 + 4 * part, lo);
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] = x[8 + i];
                        }
                    }
                } else {
                    const float bh = q > 0 ? sc->gh[32 * q - 1] : 0.f, bl = q > 0 ? sc->gl[32 * q - 1] : 0.f;
                    const float u = ex2_diff(th, tl, bh, bl);
                    const F2 u2 = f2(u, u);
                    __syncwarp();  // the last chunk's factors are read
                    for (int j = 0; j < q; ++j) {
                        const int at = 32 * j + lane;
                        v[at] = sc->dt[at] * ex2_diff(bh, bl, sc->gh[at], sc->gl[at]);
                    }
                    __syncwarp();
                    wait(bar_cb, c & 1, flag, limit);
                    tc_fence_after();
#pragma unroll 1
                    for (int j = 0; j < 2 * q; ++j) {
                        float x[16];
                        tmem_ld16(row + 16 * j, x);
                        ld_wait_for(x);
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 f = *reinterpret_cast<const float4 *>(v + 16 * j + 4 * i);
                            split2(f2(x[4 * i], x[4 * i + 1]) * u2 * f2(f.x, f.y), w[2 * i], w[8 + 2 * i]);
                            split2(f2(x[4 * i + 2], x[4 * i + 3]) * u2 * f2(f.z, f.w), w[2 * i + 1], w[8 + 2 * i + 1]);
                        }
                        tmem_st16(row + 16 * j, w);
                    }
                    const uint32_t none[16] = {};
#pragma unroll 1
                    for (int j = 2 * q + 2; j < 8; ++j) tmem_st16(row + 16 * j, none);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_m);
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
#pragma unroll 1
            for (int r = 0; r < 32; r += 8) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const size_t at = from_off + static_cast<size_t>(s_row + r + e) * NS + s_col;
                    v[e] = !from ? 0.f
                           : from_bf16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(from)[at]) << 16)
                                       : from[at];
                }
                tmem_st8f(own + r, v);
                const F2 w[4] = {f2(v[0], v[1]), f2(v[2], v[3]), f2(v[4], v[5]), f2(v[6], v[7])};
                if (!TRANS) hand_on(r, w);
            }
            tmem_st_wait();
            if (!TRANS) handed_on();
#pragma unroll 1
            for (int c = 0; c < n_chunks; ++c) {
                const bool more = !TRANS && c + 1 < n_chunks;
                wait_scal(c);
                const float decay = scal(c)->decay;
                const F2 d2 = f2(decay, decay);
                wait(bar_u, c & 1, flag, limit);
                if (more) wait(bar_cs, c & 1, flag, limit);  // the product with this chunk's S0 has read it
                tc_fence_after();
#pragma unroll 1
                for (int r = 0; r < 32; r += 8) {
                    float v[8], a[8], b[8];
                    tmem_ld8(own + r, v);
                    tmem_ld8(add + r, a);
                    tmem_ld8(add + 64 + r, b);
                    ld_wait_for(v);
                    ld_wait_for(a);
                    ld_wait_for(b);
                    F2 w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[e] = fma2(f2(v[2 * e], v[2 * e + 1]), d2, f2(a[2 * e], a[2 * e + 1]) + f2(b[2 * e], b[2 * e + 1]));
                        unpack(w[e], v[2 * e], v[2 * e + 1]);
                    }
                    tmem_st8f(own + r, v);
                    if (more) hand_on(r, w);
                }
                tmem_st_wait();
                tc_fence_before();
                if (more) handed_on();
                __syncwarp();
                if (lane == 0) mbar_arrive(u_read), mbar_arrive(scal_free + 8 * (c % kScal));
            }
#pragma unroll 1
            for (int r = 0; r < 32 && !*flag; r += 8) {
                float v[8];
                tmem_ld8(own + r, v);
                ld_wait_for(v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!finite(v[e])) marked[s_row + r + e] = 1, *redo = 1;
            }
        }
    } else if (warp < kOutWarp) {
        // ------------------------------------------------------------ steps
        const int row = tid - 32 * kStepWarp;
#pragma unroll 1
        for (int c = 0; c < n_chunks; ++c) {
            const int n = min(kL, len - c * kL);
            wait_scal(c);
            const Scal *sc = scal(c);
            const bool live = row < n;
            const float w = live ? sc->dt[row] * ex2_diff(sc->gh[kL - 1], sc->gl[kL - 1], sc->gh[row], sc->gl[row]) : 0.f;
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
                split2(pair_of(v.x) * w2, hi.x, lo.x);
                split2(pair_of(v.y) * w2, hi.y, lo.y);
                split2(pair_of(v.z) * w2, hi.z, lo.z);
                split2(pair_of(v.w) * w2, hi.w, lo.w);
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
    } else if (warp < kIssueWarp) {
        // ---------------------------------------------------------- outputs
        if (!TRANS) {
            const int q = warp - kOutWarp, t = 32 * q + lane;
            constexpr int kPasses = OF32 ? 2 : 1, kPieces = 8 / kPasses;
#pragma unroll 1
            for (int c = 0; c < n_chunks; ++c) {
                const int n = min(kL, len - c * kL);
                wait_scal(c);
                const float e = ex2_approx(scal(c)->gh[t] + scal(c)->gl[t]);
                const F2 e2 = f2(e, e);
                wait(bar_y, c & 1, flag, limit);
                tc_fence_after();
                uint8_t *const tile = base + M::oX + (c % kStagesX) * kTile;
#pragma unroll 1
                for (int pass = 0; pass < kPasses; ++pass) {
#pragma unroll 1
                    for (int i = 0; i < kPieces; ++i) {
                        const uint32_t col = 8 * (pass * kPieces + i);
                        float y[8], a[8], b[8];
                        tmem_ld8(lane_base + kColY + col, y);
                        tmem_ld8(lane_base + kColCS + col, a);
                        tmem_ld8(lane_base + kColCS + 64 + col, b);
                        ld_wait_for(y);
                        ld_wait_for(a);
                        ld_wait_for(b);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            unpack(fma2(e2, f2(a[2 * k], a[2 * k + 1]) + f2(b[2 * k], b[2 * k + 1]), f2(y[2 * k], y[2 * k + 1])),
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
                    __syncwarp();
                    if (pass == kPasses - 1 && lane == 0) mbar_arrive(y_read), mbar_arrive(scal_free + 8 * (c % kScal));
                    // four rows of 128 bytes at a time
#pragma unroll 2
                    for (int k = 0; k < 8; ++k) {
                        const int r = 32 * q + 4 * k + (lane >> 3), part = lane & 7;
                        const uint4 v = *reinterpret_cast<const uint4 *>(tile + sw128_off(r, 8 * part));
                        const size_t at = ((static_cast<size_t>(t0) + c * kL + r) * p.lv.heads + h) * p.lv.p + row0;
                        if (r < n) {
                            if (OF32) *reinterpret_cast<uint4 *>(static_cast<float *>(p.in.o) + at + 32 * pass + 4 * part) = v;
                            else *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.in.o) + at + 8 * part) = v;
                        }
                    }
                    __syncwarp();
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(empty_x + 8 * (c % kStagesX));
            }
        }
    } else if (warp == kIssueWarp) {
        // ------------------------------------------------------------ issue
        const uint64_t b_k = desc_sw128(sbase + M::oB), b_mn = desc_sw128_mn(sbase + M::oB, kTile);
        const uint64_t w_mn = desc_sw128_mn(sbase + M::oW, kTile), s_mn = desc_sw128_mn(sbase + M::oS, M::kS);
        const uint64_t c_k = desc_sw128(sbase + M::oC), x_mn = desc_sw128_mn(sbase + M::oX, 8192);
#pragma unroll 1
        for (int c = 0; c < n_chunks && !*flag; ++c) {
            const uint64_t c_st = c_k + (c % kStages) * (M::kState >> 4), x_st = x_mn + (c % kStagesX) * (kTile >> 4);
            wait(full_b, c & 1, flag, limit);
            if (!TRANS) {
                wait(full_c + 8 * (c % kStages), (c / kStages) & 1, flag, limit);
                if (len - c * kL < kL) wait(bar_w, c & 1, flag, limit);  // B's rows behind the end are zeros now
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
                umma_slices<8>(tmem + kColU, b_mn, 2048, w_mn, 2048, idesc_bf16_f32(128, 128, 1) | (1u << 15), false);
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
        if (elect_one()) umma_commit(drain);
        __syncwarp();
        if (lane == 0) mbar_wait_bounded(drain, 0, limit);
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------------------ loads
        if (lane == 0 && p.test_skip_loads != 1 && !(TRANS && p.test_skip_loads == 2)) {
            const int g = h / (p.lv.heads / p.lv.groups);
            prefetch_tensormap(&maps.x);
            prefetch_tensormap(&maps.b);
            if (!TRANS) prefetch_tensormap(&maps.c);
            int in_x = 0, in_b = 0;  // loads issued
#pragma unroll 1
            for (int c = 0; c < n_chunks; ++c) {
                const int st = c % kStages, sx = c % kStagesX, t = t0 + c * kL;
                if (!TRANS && c >= kStages) wait(empty_c + 8 * st, ((c / kStages) - 1) & 1, flag, limit);
                if (c >= kStagesX) wait(empty_x + 8 * sx, ((c / kStagesX) - 1) & 1, flag, limit);
                if (*flag) break;
                if (!TRANS) {
                    mbar_arrive_expect_tx(full_c + 8 * st, M::kState);
#pragma unroll
                    for (int k = 0; k < NS / 64; ++k)
                        tma_load_3d(sbase + M::oC + st * M::kState + k * kTile, &maps.c, 64 * k, g, t, full_c + 8 * st);
                }
                mbar_arrive_expect_tx(full_x + 8 * sx, kTile);
                tma_load_3d(sbase + M::oX + sx * kTile, &maps.x, row0, h, t, full_x + 8 * sx);
                ++in_x;
                if (c > 0) wait(bar_u, (c - 1) & 1, flag, limit);
                if (*flag) break;
                ++in_b;
                mbar_arrive_expect_tx(full_b, M::kState);
#pragma unroll
                for (int k = 0; k < NS / 64; ++k) tma_load_3d(sbase + M::oB + k * kTile, &maps.b, 64 * k, g, t, full_b);
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
        const float a2 = __ldg(p.in.a + h), bias = p.in.dt_bias ? __ldg(p.in.dt_bias + h) : 0.f;
        const bool biased = p.in.dt_bias != nullptr;
        float th = 0.f, tl = 0.f;  // the sum over this warp's chunks (TRANS)
        auto fetch = [&](int t) -> uint32_t {
            const size_t at = static_cast<size_t>((static_cast<long long>(t0) + min(t, len - 1)) * p.in.dt_stride + h);
            return p.in.dt_bf16 ? static_cast<uint32_t>(__ldg(static_cast<const unsigned short *>(p.in.dt) + at))
                                : __ldg(static_cast<const uint32_t *>(p.in.dt) + at);
        };
        auto tokens_of = [&](int c, uint32_t (&raw)[4]) {
#pragma unroll
            for (int k = 0; k < 4; ++k) raw[k] = fetch(c * kL + 32 * k + lane);
        };
        uint32_t raw[4], next[4];
        tokens_of(mine, raw);
#pragma unroll 1
        for (int c = mine; c < n_chunks; c += kScalWarps) {
            tokens_of(c + kScalWarps, next);
            if (c >= kScal) wait(scal_free + 8 * (c % kScal), ((c / kScal) - 1) & 1, flag, limit);
            __syncwarp();
            Scal *sc = scal(c);
            float bh = 0.f, bl = 0.f;  // the sum up to this run
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                const bool live = c * kL + 32 * k + lane < len;
                const float x = __uint_as_float(p.in.dt_bf16 ? raw[0] << 16 : raw[0]);
                const float y = biased ? __fadd_rn(x, bias) : x;
                const float dt = live ? p.in.softplus ? softplus(y) : y : 0.f;
                float g = live ? __fmul_rn(__fmul_rn(dt, a2), kLog2e) : 0.f, l = 0.f;
                if (g < -160.f) g = -160.f;  // (a NaN stays)
#pragma unroll 1
                for (int off = 1; off < 32; off *= 2) {
                    const float u = __shfl_up_sync(0xffffffffu, g, off), v = __shfl_up_sync(0xffffffffu, l, off);
                    if (lane >= off) pair_add(g, l, u, v);
                }
                pair_add(g, l, bh, bl);
                sc->gh[32 * k + lane] = g;
                sc->gl[32 * k + lane] = l;
                sc->dt[32 * k + lane] = dt;
                bh = __shfl_sync(0xffffffffu, g, 31), bl = __shfl_sync(0xffffffffu, l, 31);
                raw[0] = raw[1], raw[1] = raw[2], raw[2] = raw[3];
            }
            if (lane == 31) sc->decay = ex2_approx(bh + bl);
            if (TRANS) pair_add(th, tl, bh, bl);
            __syncwarp();
            if (lane == 0) mbar_arrive(scal_ready + 8 * (c % kScal));
#pragma unroll
            for (int k = 0; k < 4; ++k) raw[k] = next[k];
        }
        if (TRANS && lane == 31) total[2 * mine] = th, total[2 * mine + 1] = tl;
    }

    tc_fence_before();
    __syncthreads();
    const bool gave_up = *flag != 0;
    if (TRANS && tid == 0) {
        float gh = total[0], gl = total[1];
        pair_add(gh, gl, total[2], total[3]);
        sg.decay[unit * (sg.n - 1) + segment] = ex2_approx(gh + gl);
    }
    if (tid == 0) {
        if (gave_up) flag_status(p.lv.status, WKV7_DEV_WAIT_TIMEOUT);
        if (TRANS) sg.gave_up[unit * (sg.n - 1) + segment] = gave_up;
    }
    if (!gave_up) {
        if (store && warp >= kStateWarp && warp < kStepWarp && s_col < NS) {
#pragma unroll 1
            for (int r = 0; r < 32; r += 8) {
                float v[8];
                tmem_ld8(lane_base + kColS + s_row + r, v);
                ld_wait_for(v);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = s_row + r + e;
                    if (!marked[i]) store_out(to, to_bf16, to_off + static_cast<size_t>(i) * NS + s_col, v[e]);
                }
            }
        }
        if (*redo)  // (a segment whose state goes nowhere writes its outputs alone)
            run_by_token<NS>(p, marked, h, row0, t0, len, from, from_off, from_bf16, store ? to : nullptr, to_off, to_bf16, !TRANS);
    }
    __syncthreads();
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
    const int n = min(sg.n, (t1 - t0 + sg.tokens - 1) / sg.tokens);  // this sequence's segments
    if (n < 2) return;  // (it starts from its slot)
    const size_t unit = static_cast<size_t>(seq) * gridDim.y + blockIdx.y;
    int lost = 0;
    for (int j = 0; j < n - 1; ++j) lost |= sg.gave_up[unit * (sg.n - 1) + j];
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

// [tokens][heads][size] bf16 with rows `stride` elements apart; one box = 128 tokens x
// 1 head x 64 elements, swizzled as the tiles are, zeros past the end.
bool encode(CUtensorMap *map, const void *ptr, int size, int heads, int tokens, long long stride) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(size), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(size) * 2, static_cast<cuuint64_t>(stride) * 2};
    cuuint32_t box[3] = {64, 1, kL};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NS, bool OF32, bool TRANS>
cudaError_t launch_chunks(const SsmRunArgs &a, const Segments &sg, const Maps &maps, dim3 grid, cudaStream_t s) {
    constexpr int bytes = static_cast<int>(Smem<NS>::kBytes) + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
    auto kernel = ssm_chunk_kernel<NS, OF32, TRANS>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return e != cudaSuccess ? e : launch_pdl(kernel, grid, dim3(kThreads), bytes, s, a, sg, maps);
}

template <int NS, bool OF32>
cudaError_t chunk_as(const SsmRunArgs &a, const SsmSplit &split, cudaStream_t s, int *launches) {
    Maps maps;
    if (!encode(&maps.x, a.in.x, a.lv.p, a.lv.heads, a.total_tokens, a.in.x_stride) ||
        !encode(&maps.b, a.in.b, NS, a.lv.groups, a.total_tokens, a.in.b_stride) ||
        !encode(&maps.c, a.in.c, NS, a.lv.groups, a.total_tokens, a.in.c_stride))
        return cudaErrorInvalidValue;
    const unsigned n = static_cast<unsigned>(a.n), x = static_cast<unsigned>(a.lv.heads * (a.lv.p / 64));
    Segments sg{};
    if (split.segments < 2) {
        ++*launches;
        return launch_chunks<NS, OF32, false>(a, sg, maps, dim3(x, n < 65535u ? n : 65535u, (n + 65534u) / 65535u), s);
    }
    const size_t units = static_cast<size_t>(n) * x;
    sg.tokens = split.chunks * kL;
    sg.n = split.segments;
    sg.state = static_cast<float *>(a.workspace);
    sg.decay = sg.state + units * sg.n * (64 * NS);
    sg.gave_up = reinterpret_cast<int *>(sg.decay + units * (sg.n - 1));
    sg.lost = sg.gave_up + units * (sg.n - 1);
    const unsigned z = static_cast<unsigned>(sg.n - 1);
    cudaError_t e = launch_chunks<NS, false, true>(a, sg, maps, dim3(x, n, z), s);
    ++*launches;
    if (e != cudaSuccess) return e;
    e = launch_pdl(ssm_join_kernel<NS>, dim3(64 * NS / 4 / kJoinThreads, x, n), dim3(kJoinThreads), 0, s, a, sg);
    ++*launches;
    if (e != cudaSuccess) return e;
    ++*launches;
    return launch_chunks<NS, OF32, false>(a, sg, maps, dim3(x, n, z + 1), s);
}

}  // namespace

bool ssm_chunk_takes(const SsmRunArgs &a) {
    return a.in.bf16 && a.cu_seqlens && a.total_tokens > 0 && a.in.x_stride > 0 && a.in.b_stride > 0 && a.in.c_stride > 0;
}

SsmSplit ssm_plan_split(int n_seqs, int heads, int p, int max_seqlen) {
    SsmSplit best{};
    const long long units = static_cast<long long>(n_seqs) * heads * (p / 64);
    const int chunks = (max_seqlen + kL - 1) / kL;
    if (units <= 0 || units >= 152 || chunks < 8 || n_seqs > 65535) return best;
    constexpr double kStartUs = 8, kChunkUs = 2.2, kTransUs = 1.0, kJoinUs = 5;
    auto rounds = [](long long ctas) { return static_cast<double>((ctas + 151) / 152); };
    double least = 0.8 * (kStartUs + kChunkUs * chunks);
    for (int n = 2; n <= 128 && n * 2 <= chunks; ++n) {
        const int per = (chunks + n - 1) / n;
        if ((chunks + per - 1) / per != n) continue;
        const double t = rounds(units * (n - 1)) * (kStartUs + kTransUs * per) + kJoinUs + rounds(units * n) * (kStartUs + kChunkUs * per);
        if (t < least) {
            least = t;
            best.segments = n;
            best.chunks = per;
        }
    }
    return best;
}

size_t ssm_split_bytes(const SsmSplit &split, long long units, int ds) {
    if (split.segments < 2) return 0;
    const size_t n = static_cast<size_t>(split.segments), u = static_cast<size_t>(units);
    return (u * (n * 64 * ds + 2 * (n - 1) + 1) * 4 + 15) / 16 * 16;
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
