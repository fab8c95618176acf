// The gated delta rule over whole sequences, by chunks of 64 tokens on the tcgen05
// tensor cores.
//
// Per value head, S [dv][dk] (i value, j key), a token does
//     S <- exp(g) S;  e = beta (v - S k);  S <- S + e k^T;  o = scale S q.
// Over a chunk from state S0, with G_t the sum of the log decays up to token t and
// D_ts = exp(G_t - G_s), unrolling gives for the columns e_t
//     E = F diag(beta),  (I + A) F^T = V - diag(exp G) K S0^T,   A_ts = D_ts <k_t, k_s> beta_s, s < t
//     O   = scale (diag(exp G) Q S0^T + P F^T),                  P_ts = D_ts <q_t, k_s> beta_s, s <= t
//     S_L = exp(G_L) S0 + F diag(beta exp(G_L - G)) K
// All factors are exp of differences of G with s <= t, so at most 1: no decay is
// too strong.  G is kept as a pair of floats, so that a difference stays exact
// after a token that empties the state (g log2 e is taken as at least -160; 2^-160
// is 0 in float32).
//
// Precision.  q, k and v are bf16 and go to the tensor cores as they were loaded:
// their lengths, decays, beta and scale are float32 factors on the accumulators.
// The computed operands (S0, the right-hand sides, F, T = (I + A)^-1 and P) are
// split into two bf16 parts, 16 bits; a product of two split operands leaves out
// only lo x lo (2^-18).  States stay float32 in tensor memory from chunk to chunk.
//
// One CTA owns one (sequence, value head) and walks its chunks.  Its warps:
//   scalars (warps 20, 22)  lengths of q and k, running decays, every per-token factor
//   prep (warps 0-3)       A from K K^T and P from Q K^T
//   inverse (warps 24-27)  T, two warps for every other chunk: forward substitution in four
//                          16 x 16 blocks (float32), then T21 = -T22 A21 T11 for blocks of 16
//                          and of 32 by warp-level bf16 products of two parts
//   chain (warps 4-19)     the recurrence proper, in four products of M = dv:
//     [X_K X_Q] = S0 [K; Q]^T    N = 128, K = dk, S0 from tensor memory, in two parts
//     R = v - exp(G) / |k| X_K                               (CUDA cores)
//     F = R [T_hi; T_lo]^T       N = 128, K = 64, R from tensor memory; the halves add up
//     S += F' K                  N = dk,  K = 64, F' = F diag(..) from tensor memory
//     O = F [P_hi; P_lo]^T       N = 128, K = 64, F from tensor memory; the halves add up
//   issue (warps 23, 21)    23: the chain's MMAs; 21: TMA loads (three chunks of k and q, two
//                          of v) and the prep products
// Value rows sit in the accumulator's lanes throughout, so what one product leaves is
// the next one's A operand in the same lanes, written straight back to tensor memory;
// only T and P pass through shared memory.  All waits are bounded.
//
// A tcgen05.mma of K = 16 with A from tensor memory takes 50 cycles at N = 64, 67 at 128 and
// 132 at 256 (measured, steady), so the products are laid out for N = 128.
//
// Bound by the chain's latency: each chunk's four products wait for each other, with a pass
// through the registers of all chain warps between them, and tensor memory holds one unit an
// SM.  8 sequences of 4,096 tokens, 16 key and 32 value heads of 128: 506 us, 256 units on 152
// SMs, 4.1 us a chunk, of which the products themselves are 1.6, and 11 us for a CTA's start and
// end; half of the issue slots are busy.  Inputs, outputs and states alone, at the copy rate,
// would take 125 us.
//
// Values that are not finite.  In a product over the tokens of a chunk a zero coefficient does not
// keep a NaN or an infinity of a later token away from an earlier one, as the formulas do.  A value row
// that meets one has no finite entry in its state from the chunk's end on (F is not finite, and
// neither is F' K in any column), so that one entry of the CTA's last state shows it: such a row is
// marked, its state is not stored, and it runs through the CTA's tokens once more, one by one in
// float32 (run_by_token), over the outputs and checkpoints written.  (A look at every chunk, so that
// clean chunks need not run again, cost 1 to 4% of every call.)
//
// Few (sequence, head) units leave most SMs idle, so a long sequence is then cut into
// segments of whole chunks.  A segment maps its start state to S Phi + Psi: TRANS runs its
// recurrence without outputs, once from zero (Psi) and once without values from the
// identity (Phi, whose rows evolve like any others); gdn_join_kernel chains the segments'
// states in float32; then the ordinary kernel runs all segments side by side from them.
#include "chunk_common.cuh"
#include "device_common.cuh"
#include "gdn_internal.h"
#include "wkv7_internal.h"

#include <algorithm>
#include <cmath>

namespace wkv7 {
namespace {

constexpr int kL = 64;
// Warps: prep 0-3, chain 4-19 (four for each 32 lanes: a quarter of the columns each); 72
// registers a thread.  Warp w issues on scheduler w % 4, and the schedulers are busy half of
// the time, so the work beside the chain is dealt out evenly: prep's rows of four batches are on
// 1 and 3, so the scalars are on 0 and 2, and the inverse takes turns (8 x 4,096 tokens in whole
// sequences: 575 us with the scalars on 2 and 3 and one pair of warps for the inverse, on 0 and
// 1; 555 so).
constexpr int kThreads = 896;
constexpr int kPrepWarps = 4, kIssueWarp = 23, kLoadWarp = 21, kScalWarp = 20, kInvWarp = 24;
constexpr int kCols = 16;  // of each 64 columns, a chain thread's share
constexpr int kStagesKQ = 3, kBufs = 2, kScal = 4;
// A's 16 x 16 diagonal blocks in float32: rows of 16, their 16-byte parts rotated so that
// eight rows' writes meet no bank twice.
__device__ __forceinline__ int diag_at(int row, int col) { return row * 16 + ((col >> 2) ^ ((row >> 1) & 3)) * 4; }
// Per-token factors of a chunk (rows of 64 floats), then exp(G_L): of X_K (negative), of
// F for the state, of X_Q; beta / |k|, -G as a pair; the factors of A's and P's rows.
enum { kCx = 0, kCe, kCo, kNk, kGh, kGl, kRowA, kRowP, kScalRows };

// Tensor-memory columns (512): S float32; its bf16 parts, then (the product with them done)
// F's two halves; X_K, then F's operand; X_Q; R's operand, then F''s; O's two halves over
// those last two; prep's [K; Q] K^T.  A bf16 operand holds K elements 2c, 2c + 1 in column c.
constexpr uint32_t kColS = 0, kColSHi = 128, kColSLo = 192, kColX = 256, kColXQ = 320, kColR = 384, kColKKQ = 448;

// A split sequence's segments: `tokens` each (a multiple of 64; 0: not split); Phi of all but
// the last, [unit][n - 1][dk][dk]; and [unit][n][dv][dk], Psi of segment j at j + 1, from the
// join on the state that segment j starts from at j.  (At 0 a copy of the slot's state: the
// last segment may store its own there before the first has read it.)  A transfer CTA says in
// gave_up[unit][n - 1][2] (Psi, Phi) whether one of its waits did, and the join, which then leaves the
// unit alone, in lost[unit]: the unit's CTAs of the last pass give up in turn, and its slot keeps its state.
struct Segments {
    int tokens, n;
    int kinds;  // TRANS: 0 both, Psi and Phi in turn; 1 Psi; 2 Phi
    float *phi, *psi;
    int *gave_up, *lost;
    // The three pieces of a call that is not split, one after the other: they begin at
    // chunks 0, from1 and from2 of their sequence, piece j with the float32 state of unit u that piece j - 1 left in
    // carry[u][dv][dk] before it raised the low byte of done[u] to j.  Above that byte done[0] counts the
    // CTAs that have started, each of which takes its piece from the count: the first pieces of
    // all units first, so that whatever order CTAs are started in, the piece that one waits for is
    // done or runs.  (Pieces are taken for fewer than 20 x 152 units: see plan_pieces.)
    int from1, from2;
    float *carry;
    unsigned *done;
};

constexpr int kMaxOrder = 512;  // sequences that are put in order

struct Maps {
    CUtensorMap q, k, v;
};

// Shared memory, from the first 1024-byte boundary: tiles, then the small items.
constexpr uint32_t kTile = 8192;  // 64 rows of 128 bytes, 128-byte swizzle
// OF32: float32 outputs.  F P^T then keeps P in three parts and adds lo x lo: with
// keys that hardly differ the f_t telescope, |sum P f| is far below sum |P f|, and
// two parts left errors of 5e-5 of the largest output (200 tokens of such keys;
// three: 2.6e-5).  For bf16 outputs, which round by 2^-9, two parts of each are enough
// (F as bf16 alone, 4.8e-3 of the largest output, is not).
template <int DK, int DV, bool OF32>
struct Smem {
    static constexpr int kStagesV = OF32 ? 1 : 2;      // the third part of P takes the second one's place
    static constexpr uint32_t kTP = (OF32 ? 5 : 4) * kTile;
    static constexpr uint32_t kKQ = DK / 64 * 2 * kTile;  // per stage: for each 64 of dk, K rows then Q rows
    static constexpr uint32_t kV = DV / 64 * kTile;
    static constexpr uint32_t oKQ = 0;
    static constexpr uint32_t oV = oKQ + kStagesKQ * kKQ;
    static constexpr uint32_t oTP = oV + kStagesV * kV;  // per buffer: T hi, T lo, P hi, P lo(, P's third part): rows t, 64 columns s
    // A below its 16 x 16 diagonal blocks, per buffer: hi then lo, 32 rows each: A21 of the
    // 32 x 32 blocks in columns 0-31, those of the two pairs of 16 in columns 32-47
    static constexpr uint32_t oA = oTP + kBufs * kTP;
    static constexpr uint32_t oD = oA + kBufs * kTile;  // per buffer: the diagonal blocks, float32
    static constexpr uint32_t oScal = oD + kBufs * 4 * 256 * 4;
    static constexpr uint32_t kScalBytes = kScalRows * kL * 4 + 16;
    static constexpr uint32_t oBar = oScal + kScal * kScalBytes;
    static constexpr uint32_t kBars = 2 * kStagesKQ + 2 * kStagesV + 2 + kScal + 4 * kBufs + 10 + 2;
    static constexpr uint32_t oHold = oBar + kBars * 8;
    static constexpr uint32_t oRedo = oHold + 32;  // per value row: marked (see the file's header)
    static constexpr uint32_t kBytes = oRedo + DV;
};

__device__ __forceinline__ uint32_t round2(F2 x) {
    float a, b;
    unpack(x, a, b);
    return pack_bf16_rn(a, b);
}
// (x, y) += the squares of the low and the high bf16 of a pair.
__device__ __forceinline__ void add_squares(uint32_t pair, float &x, float &y) {
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tfma.rn.f32.bf16 %0, l, l, %0;\n\tfma.rn.f32.bf16 %1, h, h, %1;}"
        : "+f"(x), "+f"(y) : "r"(pair));
}
__device__ __forceinline__ void lds4(const float *p, F2 &a, F2 &b) {  // 16-byte aligned
    const float4 x = *reinterpret_cast<const float4 *>(p);
    a = f2(x.x, x.y);
    b = f2(x.z, x.w);
}

// A transposition among four lanes, its own inverse: part c of lane l's row (16 bytes of 64) goes
// to lane c as its part l, so that a load or store of one part by four lanes is 64 contiguous
// bytes of a row.  (A part of its own row a lane is 32 lines an instruction: the state of a head
// of 128 took 5,500 cycles to store so, 2,500 now; ragged prefill of 64 x 512 tokens 657 -> 624 us.)
__device__ __forceinline__ void exchange_pairs(F2 &a0, F2 &a1, F2 &b0, F2 &b1, int mask, bool upper) {
    unsigned long long x0 = upper ? a0.v : b0.v, x1 = upper ? a1.v : b1.v;
    x0 = __shfl_xor_sync(0xffffffffu, x0, mask);
    x1 = __shfl_xor_sync(0xffffffffu, x1, mask);
    if (upper) a0.v = x0, a1.v = x1;
    else b0.v = x0, b1.v = x1;
}
__device__ __forceinline__ void exchange4(F2 (&s)[8], int lane) {
    exchange_pairs(s[0], s[1], s[2], s[3], 1, lane & 1);
    exchange_pairs(s[4], s[5], s[6], s[7], 1, lane & 1);
    exchange_pairs(s[0], s[1], s[4], s[5], 2, lane & 2);
    exchange_pairs(s[2], s[3], s[6], s[7], 2, lane & 2);
}
__device__ __forceinline__ void exchange2(uint4 (&u)[2], int lane) {  // of two lanes, two parts
    const bool upper = lane & 1;
    uint4 x = upper ? u[0] : u[1];
    x.x = __shfl_xor_sync(0xffffffffu, x.x, 1);
    x.y = __shfl_xor_sync(0xffffffffu, x.y, 1);
    x.z = __shfl_xor_sync(0xffffffffu, x.z, 1);
    x.w = __shfl_xor_sync(0xffffffffu, x.w, 1);
    if (upper) u[0] = x;
    else u[1] = x;
}

// ------------------------------------------ warp-level products for T (bf16, two parts)
// Four 8 x 8 blocks of a 16 x 16 block at (row, col) of a swizzled tile: as they lie, or
// each transposed.  With r[] = (0,0), (0,8), (8,0), (8,8): non-transposed they are the B
// fragments (k16 n8) of rows n, columns k: {r0, r1} and {r2, r3}; transposed, the A fragment
// (m16 k16) of the transposed block.
__device__ __forceinline__ uint32_t block_addr(uint32_t tile, int row, int col, int lane) {
    return tile + sw128_off(row + (lane & 7) + ((lane & 16) ? 8 : 0), col + ((lane & 8) ? 8 : 0));
}
__device__ __forceinline__ void ldm(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldm_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void stm_t(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// acc (16 x 16 B) += (fh + fl) (bh + bl) without lo x lo, a term at a time over all
// accumulators, so that consecutive instructions do not wait for each other.
template <int B, int FIRST>
__device__ __forceinline__ void mma_terms(float (&acc)[2 * B][4], const uint32_t (&fh)[4], const uint32_t (&fl)[4],
                                          const uint32_t (&bh)[B][4], const uint32_t (&bl)[B][4]) {
#pragma unroll
    for (int term = 0; term < 3; ++term)
#pragma unroll
        for (int k = FIRST; k < B; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t(&b)[4] = term == 2 ? bl[k] : bh[k];
                mma16816(acc[2 * k + x], term == 1 ? fl : fh, b[2 * x], b[2 * x + 1]);
            }
}

// 16 columns (from n0) of T21 = -T22 (A21 T11), N x N blocks with T11 at (r0, r0) of the
// tiles t and A21 at (a_row, a_col) of the tiles a, by one warp.  It computes the transposes, M^T = T11^T A21^T and
// T21^T = -M^T T22^T, so that the accumulators of the first are the A fragments of the
// second.  Every product leaves out only lo x lo.
template <int N>
__device__ __forceinline__ void off_diagonal(uint32_t t_hi, uint32_t t_lo, uint32_t a_hi, uint32_t a_lo, int r0, int n0,
                                             int a_row, int a_col, int lane) {
    constexpr int B = N / 16;
    float m[2 * B][4] = {};
#pragma unroll
    for (int j = 0; j < B; ++j) {
        if (16 * j < n0) continue;  // above T11's diagonal
        uint32_t fh[4], fl[4];
        ldm_t(block_addr(t_hi, r0 + 16 * j, r0 + n0, lane), fh);
        ldm_t(block_addr(t_lo, r0 + 16 * j, r0 + n0, lane), fl);
        uint32_t bh[B][4], bl[B][4];
#pragma unroll
        for (int k = 0; k < B; ++k) {
            ldm(block_addr(a_hi, a_row + 16 * k, a_col + 16 * j, lane), bh[k]);
            ldm(block_addr(a_lo, a_row + 16 * k, a_col + 16 * j, lane), bl[k]);
        }
        mma_terms<B, 0>(m, fh, fl, bh, bl);
    }
    float o[2 * B][4] = {};
#pragma unroll
    for (int k = 0; k < B; ++k) {
        uint32_t fh[4], fl[4];
        split2(f2(m[2 * k][0], m[2 * k][1]), fh[0], fl[0]);
        split2(f2(m[2 * k][2], m[2 * k][3]), fh[1], fl[1]);
        split2(f2(m[2 * k + 1][0], m[2 * k + 1][1]), fh[2], fl[2]);
        split2(f2(m[2 * k + 1][2], m[2 * k + 1][3]), fh[3], fl[3]);
        uint32_t bh[B][4], bl[B][4];
#pragma unroll
        for (int i = k; i < B; ++i) {  // (zero above T22's diagonal)
            ldm(block_addr(t_hi, r0 + N + 16 * i, r0 + N + 16 * k, lane), bh[i]);
            ldm(block_addr(t_lo, r0 + N + 16 * i, r0 + N + 16 * k, lane), bl[i]);
        }
        if (k == 0) mma_terms<B, 0>(o, fh, fl, bh, bl);
        else mma_terms<B, B - 1>(o, fh, fl, bh, bl);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            split2(f2(-o[2 * i + x][0], -o[2 * i + x][1]), hi[2 * x], lo[2 * x]);
            split2(f2(-o[2 * i + x][2], -o[2 * i + x][3]), hi[2 * x + 1], lo[2 * x + 1]);
        }
        stm_t(block_addr(t_hi, r0 + N + 16 * i, r0 + n0, lane), hi);
        stm_t(block_addr(t_lo, r0 + N + 16 * i, r0 + n0, lane), lo);
    }
}

// Tokens t0 .. t0 + len - 1 of the marked value rows of one head, one by one in float32, by the first 16
// warps of a CTA.  Rare, so written to be small.
template <int DK, int DV>
__device__ __noinline__ void run_by_token(const GdnRunArgs &p, const uint8_t *marked, int h, int t0, int len, int ck0,
                                          const float *from, size_t state_off, bool from_bf16, float *to, size_t to_off,
                                          bool to_bf16) {
    constexpr int R = DV / 16, C = DK / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp >= 16) return;
    uint32_t mine = 0;
#pragma unroll
    for (int m = 0; m < R; ++m) mine |= static_cast<uint32_t>(marked[warp * R + m]) << m;
    if (mine == 0) return;
    const size_t at = static_cast<size_t>(warp * R) * DK + lane * C;
    const int hk = h / (p.lv.hv / p.lv.hk);
    const bool sb = p.lv.state_bf16;
    float s[R][C];
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const size_t x = state_off + at + m * DK + c;
            s[m][c] = from_bf16 ? __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(from)[x]) << 16) : from[x];
        }
    // a row without a finite entry at the start has none at the end, and the outputs that it was given
    uint32_t fine = 0;
#pragma unroll
    for (int m = 0; m < R; ++m) {
        bool any = false;
#pragma unroll
        for (int c = 0; c < C; ++c) any |= fabsf(s[m][c]) < __int_as_float(0x7f800000);
        if (__any_sync(0xffffffffu, any)) fine |= 1u << m;
    }
    if ((mine & fine) == 0) len = 0;
    auto store = [&](float *dst, size_t off, bool bf16) {
#pragma unroll
        for (int m = 0; m < R; ++m)
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (mine >> m & 1) store_out(dst, bf16, off + at + m * DK + c, s[m][c]);
    };
    auto sum = [](float x) {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        return x;
    };
#pragma unroll 1
    for (int t = 0; t < len; ++t) {
        const long long row = static_cast<long long>(t0) + t;
        float k[C], q[C], kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            k[c] = load1<true>(p.in.k, row * p.in.k_stride + hk * DK + lane * C + c);
            q[c] = load1<true>(p.in.q, row * p.in.q_stride + hk * DK + lane * C + c);
            kk = fmaf(k[c], k[c], kk), qq = fmaf(q[c], q[c], qq), kq = fmaf(k[c], q[c], kq);
        }
        const float alpha = expf(__ldg(p.in.g + row * p.in.g_stride + h)), beta = __ldg(p.in.beta + row * p.in.beta_stride + h);
        const float nk = p.in.eps > 0.f ? rsqrtf(sum(kk) + p.in.eps) : 1.f;
        const float nq = p.in.eps > 0.f ? p.in.scale * rsqrtf(sum(qq) + p.in.eps) : p.in.scale;
        kq = nk * sum(kq);
#pragma unroll
        for (int m = 0; m < R; ++m) {
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) a = fmaf(s[m][c], k[c], a), b = fmaf(s[m][c], q[c], b);
            const int i = warp * R + m;
            const float v = load1<true>(p.in.v, row * p.in.v_stride + static_cast<long long>(h) * DV + i);
            const float e = beta * (v - alpha * nk * sum(a));
            const float o = nq * fmaf(alpha, sum(b), e * kq);
#pragma unroll
            for (int c = 0; c < C; ++c) s[m][c] = fmaf(alpha, s[m][c], e * nk * k[c]);
            if (lane == 0 && (mine >> m & 1)) store_out(p.in.o, p.in.o_bf16, (static_cast<size_t>(row) * p.lv.hv + h) * DV + i, o);
        }
        if (p.cu_ckpt && (t + 1) % kL == 0) {
            if (sb) {  // the carry goes on from what a checkpoint stores
#pragma unroll
                for (int m = 0; m < R; ++m)
#pragma unroll
                    for (int c = 0; c < C; ++c) s[m][c] = round_bf16(s[m][c]);
            }
            const int id = __ldg(p.ckpt_ids + ck0 + t / kL);
            if (id >= 0 && id < p.lv.n_snaps)  // (flagged before)
                store(p.lv.snaps, static_cast<size_t>(id) * p.lv.slot_stride + p.lv.layer_off + static_cast<size_t>(h) * DV * DK, sb);
        }
    }
    if (to) store(to, to_off, to_bf16);
}

enum Mode { kWhole, kTransfer, kPiece };  // whole sequences or segments; segments' Psi and Phi; pieces

template <int DK, int DV, bool OF32, Mode MODE>
__global__ void __launch_bounds__(kThreads, 1)
    gdn_chunk_kernel(const __grid_constant__ GdnRunArgs p, const Segments sg, const __grid_constant__ Maps maps) {
    using M = Smem<DK, DV, OF32>;
    constexpr bool TRANS = MODE == kTransfer, PIECES = MODE == kPiece;
    constexpr int kStagesV = M::kStagesV;
    constexpr int kChainWarps = DV / 8;  // with something to do
    extern __shared__ uint8_t smem_raw[];
    pdl_prologue();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int h = blockIdx.x, seq = blockIdx.y + (PIECES || sg.tokens ? 0 : blockIdx.z * 65535), piece = 0;
    if (seq >= p.n) return;
    unsigned *const drawn = reinterpret_cast<unsigned *>(smem_raw) + kMaxOrder + 4;
    if (PIECES && tid == 0) *drawn = atomicAdd(sg.done, 256u) >> 8;
    auto take_piece = [&] {  // after a barrier
        const unsigned at = *drawn, heads = p.lv.hv, unit = at % (heads * p.n);
        piece = at / (heads * p.n), seq = unit / heads, h = unit % heads;
    };
    int slot, t0, t1;
    if ((PIECES || !sg.tokens) && p.n > 1 && p.n <= kMaxOrder) {  // the longest sequences start first: their ends are not the grid's
        int *key = reinterpret_cast<int *>(smem_raw);
        int4 *found = reinterpret_cast<int4 *>(key + kMaxOrder);
        int4 mine{};  // of sequence tid
        if (tid < p.n) {
            mine = make_int4(tid, __ldg(p.slot_ids + tid), __ldg(p.cu_seqlens + tid), __ldg(p.cu_seqlens + tid + 1));
            key[tid] = (mine.w - mine.z + kL - 1) / kL;
        }
        __syncthreads();
        if (PIECES) take_piece();
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
        if (PIECES) {
            __syncthreads();
            take_piece();
            __syncthreads();
        }
        slot = __ldg(p.slot_ids + seq), t0 = __ldg(p.cu_seqlens + seq), t1 = __ldg(p.cu_seqlens + seq + 1);
    }
    if (slot < 0 || slot >= p.lv.n_slots) {
        if (tid == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SLOT);
        return;
    }
    bool bad = t0 < 0 || t1 < t0 || t1 > p.total_tokens || t1 - t0 > p.max_seqlen;
    int ck0 = 0;
    if (!bad && p.cu_ckpt) {
        ck0 = __ldg(p.cu_ckpt + seq);
        bad = ck0 < 0 || __ldg(p.cu_ckpt + seq + 1) - ck0 != (t1 - t0) / kL;
    }
    if (bad) {
        if (tid == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SEQLENS);
        return;
    }
    // this CTA's part of the sequence, and where its state comes from and goes to
    bool phi = false, to_pool = !TRANS;
    const float *from = p.lv.states;  // (null: zeros, or the identity)
    float *to = p.lv.states;
    bool from_bf16 = p.lv.state_bf16;
    int lost = 0;  // the start state: a transfer gave up
    int *gave_up = nullptr;
    size_t state_off = static_cast<size_t>(slot) * p.lv.slot_stride + p.lv.layer_off + static_cast<size_t>(h) * DV * DK;
    size_t to_off = state_off;
    if (!PIECES && sg.tokens) {
        const int z = blockIdx.z, j = TRANS && sg.kinds == 0 ? z >> 1 : z;
        phi = TRANS && (sg.kinds == 0 ? (z & 1) != 0 : sg.kinds == 2);
        const int end = t1;
        if (j > 0 && t1 - t0 <= static_cast<long long>(j) * sg.tokens) return;
        t0 += j * sg.tokens;
        t1 = min(t1, t0 + sg.tokens);
        const size_t unit = static_cast<size_t>(seq) * p.lv.hv + h;
        if (TRANS) {
            if (t1 == end) return;
            from = nullptr;
            to = phi ? sg.phi : sg.psi;
            to_off = (phi ? unit * (sg.n - 1) + j : unit * sg.n + j + 1) * (DV * DK);  // (DV is dk for Phi)
            gave_up = sg.gave_up + (unit * (sg.n - 1) + j) * 2 + phi;
        } else {
            to_pool = t1 == end;
            if (j > 0 || !to_pool) {
                from = sg.psi;
                from_bf16 = false;
                state_off = (unit * sg.n + j) * (DV * DK);
                lost = sg.lost[unit];
            }
        }
    }
    const int done_at = seq * p.lv.hv + h;  // (PIECES: of a few thousand)
    if (PIECES) {
        const int end = t1, chunks = (end - t0 + kL - 1) / kL;
        const int at = piece == 0 ? 0 : piece == 1 ? sg.from1 : sg.from2;
        const int next = piece == 0 ? sg.from1 : piece == 1 ? sg.from2 : chunks;
        if (at > 0 && chunks <= at) return;
        if (next < chunks) t1 = t0 + kL * next;
        t0 += kL * at;
        ck0 += at;
        const size_t carried = (static_cast<size_t>(seq) * p.lv.hv + h) * (DV * DK);
        if (piece > 0) from = sg.carry, from_bf16 = false, state_off = carried;
        to_pool = t1 == end;
        if (!to_pool) to = sg.carry, to_off = carried;
    }
    const int len = t1 - t0;
    if (len == 0) return;
    const int n_chunks = (len + kL - 1) / kL;

    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(base);
    volatile int *flag = reinterpret_cast<volatile int *>(base + M::oHold + 4);
    uint32_t nbar = sbase + M::oBar;
    auto bars = [&nbar](int n) { const uint32_t b = nbar; nbar += 8 * n; return b; };
    const uint32_t full_kq = bars(kStagesKQ), kq_empty = bars(kStagesKQ), full_v = bars(kStagesV), v_empty = bars(kStagesV);
    const uint32_t kkq_full = bars(1), kkq_free = bars(1), scal_ready = bars(kScal), prep_ready = bars(kBufs);
    const uint32_t a_ready = bars(kBufs), a_free = bars(kBufs);
    const uint32_t buf_free = bars(kBufs), bar_x = bars(1), bar_rhs = bars(1), bar_e = bars(1), bar_ep = bars(1);
    const uint32_t bar_eo = bars(1), bar_s = bars(1), bar_o = bars(1), s_ready = bars(2), o_read = bars(1);
    const uint32_t drain = bars(2);
    const long long limit = p.wait_cycles;
    // A piece's head is kept in shared memory: as a register of every role it spills others (8 x 4,096
    // tokens 526 us, 507 so; a grid coordinate is read where it is needed).
    volatile int *const held = reinterpret_cast<volatile int *>(base + M::oHold + 8);
    volatile int *const redo = held + 2;  // some row is marked
    uint8_t *const marked = base + M::oRedo;
    auto head = [held] { return PIECES ? held[0] : static_cast<int>(blockIdx.x); };

    if (warp == 0) tmem_alloc(sbase + M::oHold, 512);
    if (tid == 32) {
        for (int i = 0; i < kStagesKQ; ++i) mbar_init(full_kq + 8 * i, 1), mbar_init(kq_empty + 8 * i, 1);
        for (int i = 0; i < kStagesV; ++i) mbar_init(full_v + 8 * i, 1), mbar_init(v_empty + 8 * i, kChainWarps);
        for (int i = 0; i < kScal; ++i) mbar_init(scal_ready + 8 * i, 2);
        for (int i = 0; i < kBufs; ++i) mbar_init(a_ready + 8 * i, 2), mbar_init(a_free + 8 * i, 2);
        for (int i = 0; i < kBufs; ++i) mbar_init(prep_ready + 8 * i, 4), mbar_init(buf_free + 8 * i, kChainWarps);
        mbar_init(kkq_full, 1), mbar_init(kkq_free, kPrepWarps);
        mbar_init(bar_x, 1), mbar_init(bar_e, 1), mbar_init(bar_s, 1), mbar_init(bar_o, 1);
        mbar_init(bar_rhs, kChainWarps), mbar_init(bar_ep, kChainWarps), mbar_init(bar_eo, kChainWarps);
        mbar_init(s_ready, kChainWarps), mbar_init(s_ready + 8, kChainWarps), mbar_init(o_read, kChainWarps);
        mbar_init(drain, 1), mbar_init(drain + 8, 1);
        fence_mbar_init();
        *flag = lost, *redo = 0;
        if (PIECES) held[0] = h, held[1] = done_at;
        if (PIECES && piece > 0) {  // the piece before: of a CTA that started earlier, mostly long gone
            const long long since = clock64();
            int at;
            do {
                asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(at) : "l"(sg.done + done_at) : "memory");
                at &= 255;
                if (at < piece) __nanosleep(200);
            } while (at < piece && clock64() - since <= limit);
            if (at < piece) *flag = 1;
        }
    }
    if (tid < DV) marked[tid] = 0;
    // T and P are lower triangular: what lies above their 16 x 16 diagonal blocks stays zero
    for (uint32_t e = tid; e < kBufs * M::kTP / 16; e += kThreads)
        reinterpret_cast<uint4 *>(base + M::oTP)[e] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(base + M::oHold);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    // a chunk's per-token factors; a table is written again four chunks on, when k's tile is
    // free of the third: chain and prep have left the first
    auto scal = [base](int c) { return reinterpret_cast<float *>(base + M::oScal + (c % kScal) * M::kScalBytes); };

    if (warp < kPrepWarps) {
        // ------------------------------------------------------------- prep
        // Thread m: row t of A (from K) for warps 0 and 1, of P (from Q) for 2 and 3.
        // (After a wait gave up this role's and the other warps' loops run on, on whatever they
        // find: the warps of a named barrier must all come to it, and no wait holds them any more.)
        const int t = tid & 63;
        const bool is_q = tid >= 64;
        const int batches = (warp & 1) ? 4 : 2;  // of 16 columns: rows below 32 end at column 31
        for (int c = 0; c < n_chunks; ++c) {
            const int n = min(kL, len - c * kL);
            const float *sc = scal(c);
            uint8_t *tp = base + M::oTP + (c % kBufs) * M::kTP;
            wait<true>(scal_ready + 8 * (c % kScal), (c / kScal) & 1, flag, limit);
            wait<true>((is_q ? buf_free : a_free) + 8 * (c % kBufs), ((c / kBufs) & 1) ^ 1, flag, limit);
            uint8_t *A = base + M::oA + (c % kBufs) * kTile;
            float *D = reinterpret_cast<float *>(base + M::oD) + (c % kBufs) * 4 * 256;
            const float gh = -sc[kGh * kL + t], gl = -sc[kGl * kL + t], row_c = sc[(is_q ? kRowP : kRowA) * kL + t];
            const F2 gh2 = f2(gh, gh), gl2 = f2(gl, gl), rc2 = f2(row_c, row_c);
            wait<true>(kkq_full, c & 1, flag, limit);
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < (TRANS && is_q ? 0 : batches); ++b) {
                const int s = 16 * b;
                float x[16];
                tmem_ld16(lane_base + kColKKQ + s, x);
                F2 f[8];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    F2 hs[2], ls[2], ks[2];
                    lds4(sc + kGh * kL + s + 2 * e, hs[0], hs[1]);
                    lds4(sc + kGl * kL + s + 2 * e, ls[0], ls[1]);
                    lds4(sc + kNk * kL + s + 2 * e, ks[0], ks[1]);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        float d0, d1;
                        unpack((gh2 + hs[z]) + (gl2 + ls[z]), d0, d1);
                        f[e + z] = (rc2 * ks[z]) * f2(ex2_approx(d0), ex2_approx(d1));
                    }
                }
                ld_wait_for(x);
                const int keep = is_q ? t + 1 - s : (t < n ? t - s : 0);  // of this batch's columns
                float y[16];
#pragma unroll
                for (int e = 0; e < 8; ++e) unpack(f[e] * f2(x[2 * e], x[2 * e + 1]), y[2 * e], y[2 * e + 1]);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (e >= keep) y[e] = 0.f;
                if (!is_q && b == t >> 4) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<float4 *>(D + 256 * b + diag_at(t & 15, e)) =
                            make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                } else if (is_q || b < t >> 4) {
                    uint8_t *hi_tile = is_q ? tp + 2 * kTile : A;
                    const uint32_t lo_at = is_q ? kTile : kTile / 2;
                    const bool pair = !is_q && b == (t >> 5) * 2;  // below a 16-block of the same 32
                    const int row = is_q ? t : pair ? (t & 15) + 16 * (t >> 5) : t - 32, col = pair ? 32 : s;
#pragma unroll
                    for (int g = 0; g < 16; g += 8) {
                        uint32_t hi[4], lo[4];
                        const uint32_t off = sw128_off(row, col + g);
#pragma unroll
                        for (int e = 0; e < 4; ++e) split2(f2(y[g + 2 * e], y[g + 2 * e + 1]), hi[e], lo[e]);
                        *reinterpret_cast<uint4 *>(hi_tile + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4 *>(hi_tile + lo_at + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        if (OF32 && is_q) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = pack_bf16_rn((y[g + 2 * e] - bf16_lo(hi[e])) - bf16_lo(lo[e]),
                                                    (y[g + 2 * e + 1] - bf16_hi(hi[e])) - bf16_hi(lo[e]));
                            *reinterpret_cast<uint4 *>(tp + 4 * kTile + off) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(kkq_free);

            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive((is_q ? prep_ready : a_ready) + 8 * (c % kBufs));
        }
    } else if (warp < kScalWarp) {
        // ------------------------------------------------------------ chain
        // (with DV = 64 the accumulators' upper lanes hold nothing and their warps have nothing to do)
        const int i = 32 * (warp & 3) + lane;                    // value row
        const int col0 = kCols * ((warp - kPrepWarps) >> 2);     // first of this thread's columns of each 64
        if (i < DV) {
            const size_t row_off = static_cast<size_t>(i) * DK + col0;
            const bool sb = p.lv.state_bf16;

            // this thread's columns as a bf16 operand: hi parts from column `hi`, lo parts from `lo`
            auto put_operand = [&](const F2 (&x)[8], uint32_t hi_col, uint32_t lo_col) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) split2(x[e], hi[e], lo[e]);
                tmem_st8(lane_base + hi_col + col0 / 2, hi);
                tmem_st8(lane_base + lo_col + col0 / 2, lo);
            };
            // a state row part (of the b-th 64 key columns): its operand, and float32 times the chunk's decay
            auto put_state = [&](const F2 (&s)[8], int b, float decay) {
                put_operand(s, kColSHi + 32 * b, kColSLo + 32 * b);
                uint32_t f[16];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float x, y;
                    unpack(s[e] * f2(decay, decay), x, y);
                    f[2 * e] = __float_as_uint(x);
                    f[2 * e + 1] = __float_as_uint(y);
                }
                tmem_st16(lane_base + kColS + 64 * b + col0, f);
            };
            // 16 key columns of the warp's 32 value rows at dst + off (the offset of this thread's
            // own row), four lanes (bf16: two) to a row, but for the rows of the lanes in `skip`
            auto write_state = [&](float *dst, size_t off, bool bf16, F2 (&s)[8], uint32_t skip) {
                if (bf16) {
                    uint4 u[2] = {make_uint4(round2(s[0]), round2(s[1]), round2(s[2]), round2(s[3])),
                                  make_uint4(round2(s[4]), round2(s[5]), round2(s[6]), round2(s[7]))};
                    exchange2(u, lane);
                    uint16_t *d = reinterpret_cast<uint16_t *>(dst) + off - (lane & 1) * DK + 8 * (lane & 1);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (!(skip >> ((lane & ~1) + k) & 1)) *reinterpret_cast<uint4 *>(d + k * DK) = u[k];
                } else {
                    exchange4(s, lane);
                    float *d = dst + off - (lane & 3) * DK + 4 * (lane & 3);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float4 y;
                        unpack(s[2 * k], y.x, y.y);
                        unpack(s[2 * k + 1], y.z, y.w);
                        if (!(skip >> ((lane & ~3) + k) & 1)) *reinterpret_cast<float4 *>(d + k * DK) = y;
                    }
                }
            };
            auto load_cols = [&](uint32_t col, F2 (&x)[8]) {
                float v[16];
                tmem_ld16(lane_base + col + col0, v);
                ld_wait_for(v);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = f2(v[2 * e], v[2 * e + 1]);
            };
            auto signal = [&](uint32_t bar) {  // this warp's tensor-memory accesses before, the issuer's MMAs after
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
            };

            wait(scal_ready, 0, flag, limit);
            const float first_decay = scal(0)[kScalRows * kL];
#pragma unroll 1
            for (int b = 0; b < DK / 64; ++b) {
                F2 s[8];
                if (TRANS) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int c = 64 * b + col0 + 2 * e;
                        s[e] = f2(phi && c == i ? 1.f : 0.f, phi && c + 1 == i ? 1.f : 0.f);
                    }
                } else if (from_bf16) {
                    const uint16_t *src = reinterpret_cast<const uint16_t *>(from) + state_off + row_off + 64 * b -
                                          (lane & 1) * DK + 8 * (lane & 1);
                    uint4 u[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) u[k] = *reinterpret_cast<const uint4 *>(src + k * DK);
                    exchange2(u, lane);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        s[4 * k] = f2_bf16(u[k].x), s[4 * k + 1] = f2_bf16(u[k].y);
                        s[4 * k + 2] = f2_bf16(u[k].z), s[4 * k + 3] = f2_bf16(u[k].w);
                    }
                } else {
                    const float *src = from + state_off + row_off + 64 * b - (lane & 3) * DK + 4 * (lane & 3);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 u = *reinterpret_cast<const float4 *>(src + k * DK);
                        s[2 * k] = f2(u.x, u.y), s[2 * k + 1] = f2(u.z, u.w);
                    }
                    exchange4(s, lane);
                }
                put_state(s, b, first_decay);
                tmem_st_wait();
                signal(s_ready + 8 * b);
            }
            // a chunk's outputs leave while the next one's F product runs: bf16 pairs (or float32), token columns
            constexpr int kOut = OF32 ? 16 : 8;
            uint32_t out[kOut];
            auto store_out_rows = [&](int c) {
                const int n = min(kL, len - c * kL);
                if constexpr (OF32) {
                    const size_t step = static_cast<size_t>(p.lv.hv) * DV;
                    float *dst = static_cast<float *>(p.in.o) + (static_cast<size_t>(t0) + c * kL + col0) * step +
                                 static_cast<size_t>(head()) * DV + i;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        if (col0 + e < n) *dst = __uint_as_float(out[e]);
                        dst += step;
                    }
                } else {  // through 1 KB of the chunk's v tile (every warp has read its v: F depends on it), 16 bytes a lane
                    uint8_t *ot = base + M::oV + (c % kStagesV) * M::kV + ((warp & 3) + DV / 32 * (col0 / kCols)) * 1024;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {  // [16 tokens][32 value rows]
                        reinterpret_cast<uint16_t *>(ot)[2 * e * 32 + lane] = static_cast<uint16_t>(out[e]);
                        reinterpret_cast<uint16_t *>(ot)[(2 * e + 1) * 32 + lane] = static_cast<uint16_t>(out[e] >> 16);
                    }
                    __syncwarp();
                    const int t = col0 + lane / 4;
                    uint16_t *dst = static_cast<uint16_t *>(p.in.o) +
                                    ((static_cast<size_t>(t0) + c * kL + t) * p.lv.hv + head()) * DV + 32 * (warp & 3) + (lane & 3) * 8;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(ot + r * 512 + lane * 16);
                        if (t + 8 * r < n) *reinterpret_cast<uint4 *>(dst + static_cast<size_t>(8 * r) * p.lv.hv * DV) = u;
                    }
                    fence_proxy_async_smem();  // the tile's next writer is a TMA load
                    __syncwarp();
                    if (lane == 0) mbar_arrive(v_empty + 8 * (c % kStagesV));
                }
            };

#pragma unroll 1
            for (int c = 0; c < n_chunks; ++c) {
                const int n = min(kL, len - c * kL);
                const uint32_t ph = c & 1;
                const float *sc = scal(c) + col0;
                // R = v - cx X_K, v loaded while the product runs
                wait(full_v + 8 * (c % kStagesV), (c / kStagesV) & 1, flag, limit);
                F2 x[8], y[8], xq[8];
                {
                    const uint8_t *at = base + M::oV + (c % kStagesV) * M::kV + (i >> 6) * kTile;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint16_t a = *reinterpret_cast<const uint16_t *>(at + sw128_off(col0 + 2 * e, i & 63));
                        const uint16_t b = *reinterpret_cast<const uint16_t *>(at + sw128_off(col0 + 2 * e + 1, i & 63));
                        y[e] = f2(__uint_as_float(static_cast<uint32_t>(a) << 16), __uint_as_float(static_cast<uint32_t>(b) << 16));
                        if (TRANS && phi) y[e] = f2(0.f, 0.f);
                    }
                }
                wait(bar_x, ph, flag, limit);
                tc_fence_after();
                load_cols(kColX, x);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    F2 f, g;
                    lds4(sc + kCx * kL + 2 * e, f, g);
                    x[e] = fma2(f, x[e], y[e]);
                    x[e + 1] = fma2(g, x[e + 1], y[e + 1]);
                }
                if (n < kL) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float a, b;
                        unpack(x[e], a, b);
                        x[e] = f2(col0 + 2 * e < n ? a : 0.f, col0 + 2 * e + 1 < n ? b : 0.f);
                    }
                }
                put_operand(x, kColR, kColR + 32);
                tmem_st_wait();
                signal(bar_rhs);
                if ((OF32 || TRANS) && lane == 0) mbar_arrive(v_empty + 8 * (c % kStagesV));
                if (!TRANS && c > 0) store_out_rows(c - 1);

                // F, and F' = F ce for the state
                wait(bar_e, ph, flag, limit);
                tc_fence_after();
                load_cols(kColSHi, x);
                load_cols(kColSLo, y);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    F2 f, g;
                    lds4(sc + kCe * kL + 2 * e, f, g);
                    x[e] = x[e] + y[e];
                    x[e + 1] = x[e + 1] + y[e + 1];
                    y[e] = f * x[e];
                    y[e + 1] = g * x[e + 1];
                }
                put_operand(y, kColR, kColR + 32);
                tmem_st_wait();
                signal(bar_ep);
                if constexpr (TRANS) {
                    if (lane == 0) mbar_arrive(buf_free + 8 * (c % kBufs));  // T is read: E followed from it
                } else {
                    put_operand(x, kColX, kColX + 32);
                    load_cols(kColXQ, xq);
                    tmem_st_wait();
                    signal(bar_eo);
                }

                // the new state, 64 key columns at a time
                const bool last = c + 1 == n_chunks;
                const bool boundary = !TRANS && p.cu_ckpt && n == kL;
                int ck = -1;
                if (boundary) {
                    ck = __ldg(p.ckpt_ids + ck0 + c);
                    if (ck < 0 || ck >= p.lv.n_snaps) {
                        if (tid == 32 * kPrepWarps) flag_status(p.lv.status, WKV7_DEV_BAD_SLOT);
                        ck = -1;
                    }
                }
                if (!last) wait(scal_ready + 8 * ((c + 1) % kScal), ((c + 1) / kScal) & 1, flag, limit);
                const float decay = last ? 0.f : scal(c + 1)[kScalRows * kL];
                wait(bar_s, ph, flag, limit);
                tc_fence_after();
#pragma unroll 1
                for (int b = 0; b < DK / 64; ++b) {
                    load_cols(kColS + 64 * b, x);
                    if (boundary) {
                        if (sb) {  // the carry goes on from what a checkpoint stores
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = f2_bf16(round2(x[e]));
                        }
                        if (ck >= 0 && !*flag) {
                            F2 kept[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) kept[e] = x[e];
                            write_state(p.lv.snaps,
                                        static_cast<size_t>(ck) * p.lv.slot_stride + p.lv.layer_off +
                                            static_cast<size_t>(head()) * DV * DK + row_off + 64 * b,
                                        sb, kept, 0);
                        }
                    }
                    if (!last) {
                        put_state(x, b, decay);
                        tmem_st_wait();
                    } else {
                        if (!TRANS && b == 0) {
                            float first, second;
                            unpack(x[0], first, second);
                            if (!(fabsf(first) < __int_as_float(0x7f800000))) marked[i] = 1, *redo = 1;
                            bar_sync_named(1, 32 * kChainWarps);  // a row's four threads store all of it or nothing
                        }
                        if ((TRANS || PIECES || to_pool) && !*flag)
                            write_state(to, to_off + row_off + 64 * b, !TRANS && to_pool && sb, x,
                                        TRANS ? 0 : __ballot_sync(0xffffffffu, marked[i]));
                    }
                    signal(s_ready + 8 * b);
                }

                if constexpr (TRANS) continue;
                // the outputs, O = co X_Q + F P^T, while the next X is made
                wait(bar_o, ph, flag, limit);
                tc_fence_after();
                load_cols(kColXQ, x);
                load_cols(kColR, y);
                signal(o_read);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    F2 f, g;
                    lds4(sc + kCo * kL + 2 * e, f, g);
                    x[e] = fma2(f, xq[e], x[e] + y[e]);
                    x[e + 1] = fma2(g, xq[e + 1], x[e + 1] + y[e + 1]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (OF32) {
                        float a, b;
                        unpack(x[e], a, b);
                        out[2 * e] = __float_as_uint(a);
                        out[2 * e + 1] = __float_as_uint(b);
                    } else {
                        out[e] = round2(x[e]);
                    }
                }
                if (lane == 0) mbar_arrive(buf_free + 8 * (c % kBufs));
            }
            if (!TRANS) store_out_rows(n_chunks - 1);
        }
    } else if (warp == kIssueWarp) {
        // -------------------------------------------------- the chain's MMAs
        if (lane == 0) {
            for (int c = 0; c < n_chunks; ++c) {
                if (*flag) break;
                const uint32_t ph = c & 1;
                const uint32_t kq = sbase + M::oKQ + (c % kStagesKQ) * M::kKQ;
                const uint32_t tp = sbase + M::oTP + (c % kBufs) * M::kTP;
                wait(full_kq + 8 * (c % kStagesKQ), (c / kStagesKQ) & 1, flag, limit);
                if (!TRANS && c > 0) wait(o_read, ph ^ 1, flag, limit);  // X takes the columns of the last chunk's O and its operand
#pragma unroll
                for (int hh = 0; hh < DK / 64; ++hh) {  // X, as the state's halves arrive
                    wait(s_ready + 8 * hh, ph, flag, limit);
                    if (*flag) break;
                    tc_fence_after();
                    umma_ta_128xNx64(tmem + kColX, tmem + kColSHi + 32 * hh, kq + hh * 2 * kTile, 128, hh > 0, false);
                    umma_ta_128xNx64(tmem + kColX, tmem + kColSLo + 32 * hh, kq + hh * 2 * kTile, 128, true, false);
                }
                umma_commit(bar_x);
                wait(prep_ready + 8 * (c % kBufs), (c / kBufs) & 1, flag, limit);
                wait(bar_rhs, ph, flag, limit);
                if (*flag) break;
                tc_fence_after();
                umma_ta_128xNx64(tmem + kColSHi, tmem + kColR, tp, 128, false, false);
                umma_ta_128xNx64(tmem + kColSHi, tmem + kColR + 32, tp, 128, true, false);
                umma_commit(bar_e);
                wait(bar_ep, ph, flag, limit);
                if (*flag) break;
                tc_fence_after();
                umma_ta_128xNx64(tmem + kColS, tmem + kColR, kq, DK, true, true, 2 * kTile);
                umma_ta_128xNx64(tmem + kColS, tmem + kColR + 32, kq, DK, true, true, 2 * kTile);
                umma_commit(bar_s);
                umma_commit(kq_empty + 8 * (c % kStagesKQ));
                if constexpr (TRANS) continue;
                wait(bar_eo, ph, flag, limit);
                wait(bar_s, ph, flag, limit);  // O takes the columns of that product's operand
                if (*flag) break;
                tc_fence_after();
                umma_ta_128xNx64(tmem + kColXQ, tmem + kColX, tp + 2 * kTile, 128, false, false);
                umma_ta_128xNx64(tmem + kColXQ, tmem + kColX + 32, tp + 2 * kTile, 128, true, false);
                if constexpr (OF32) umma_ta_128xNx64(tmem + kColXQ, tmem + kColX, tp + 4 * kTile, 64, true, false);
                umma_commit(bar_o);
            }
            if (*flag) {  // let what was issued end before the tensor memory goes
                umma_commit(drain);
                mbar_wait_bounded(drain, 0, limit);
            }
        }
    } else if (warp == kLoadWarp) {
        // ------------------------------- input loads and the products for prep
        if (lane == 0) {
            const int h = head(), hk = h / (p.lv.hv / p.lv.hk);
            int kq_next = 0, v_next = 0, mma_next = 0;
            long long since = clock64();
            const int n_load = p.test_skip_loads == 1 || (TRANS && p.test_skip_loads) ? 0 : n_chunks;
            while (kq_next < n_load || v_next < n_load || mma_next < n_chunks) {
                bool moved = false;
                if (kq_next < n_load && mbar_try_wait(kq_empty + 8 * (kq_next % kStagesKQ), ((kq_next / kStagesKQ) & 1) ^ 1)) {
                    const int sk = kq_next % kStagesKQ, at = t0 + kq_next * kL;
                    const uint32_t kq = sbase + M::oKQ + sk * M::kKQ;
                    mbar_arrive_expect_tx(full_kq + 8 * sk, M::kKQ);
                    for (int hh = 0; hh < DK / 64; ++hh) {
                        tma_load_3d(kq + hh * 2 * kTile, &maps.k, 64 * hh, hk, at, full_kq + 8 * sk);
                        tma_load_3d(kq + hh * 2 * kTile + kTile, &maps.q, 64 * hh, hk, at, full_kq + 8 * sk);
                    }
                    ++kq_next;
                    moved = true;
                }
                if (v_next < n_load && mbar_try_wait(v_empty + 8 * (v_next % kStagesV), ((v_next / kStagesV) & 1) ^ 1)) {
                    const int sv = v_next % kStagesV;
                    mbar_arrive_expect_tx(full_v + 8 * sv, M::kV);
                    for (int hh = 0; hh < DV / 64; ++hh)
                        tma_load_3d(sbase + M::oV + sv * M::kV + hh * kTile, &maps.v, 64 * hh, h, t0 + v_next * kL, full_v + 8 * sv);
                    ++v_next;
                    moved = true;
                }
                if (mma_next < n_chunks && mbar_try_wait(full_kq + 8 * (mma_next % kStagesKQ), (mma_next / kStagesKQ) & 1) &&
                    mbar_try_wait(kkq_free, (mma_next & 1) ^ 1)) {
                    tc_fence_after();
                    const uint32_t kq = sbase + M::oKQ + (mma_next % kStagesKQ) * M::kKQ;
                    for (int hh = 0; hh < DK / 64; ++hh)
                        umma_128xNx64(tmem + kColKKQ, kq + hh * 2 * kTile, kq + hh * 2 * kTile, 64, hh > 0);
                    umma_commit(kkq_full);
                    ++mma_next;
                    moved = true;
                }
                if (*flag) break;
                if (moved) {
                    since = clock64();
                } else {
                    if (clock64() - since > limit) *flag = 1;
                    __nanosleep(200);
                }
            }
            if (*flag) {  // let what was issued end: the copies in flight and the products
                for (int c = max(0, kq_next - kStagesKQ); c < kq_next; ++c)
                    mbar_wait_bounded(full_kq + 8 * (c % kStagesKQ), (c / kStagesKQ) & 1, limit);
                for (int c = max(0, v_next - kStagesV); c < v_next; ++c)
                    mbar_wait_bounded(full_v + 8 * (c % kStagesV), (c / kStagesV) & 1, limit);
                umma_commit(drain + 8);
                mbar_wait_bounded(drain + 8, 0, limit);
            }
        }
    } else if (warp >= kInvWarp) {
        // -------------------------------------------- the inverse, T = (I + A)^-1
        const int w = warp & 1;
        for (int c = (warp - kInvWarp) >> 1; c < n_chunks; c += 2) {  // a pair of warps every other chunk
            uint8_t *tp = base + M::oTP + (c % kBufs) * M::kTP;
            const int blk = 2 * w + (lane >> 4), col = lane & 15;
            const float *d = reinterpret_cast<const float *>(base + M::oD) + ((c % kBufs) * 4 + blk) * 256;
            wait<true>(buf_free + 8 * (c % kBufs), ((c / kBufs) & 1) ^ 1, flag, limit);
            wait<true>(a_ready + 8 * (c % kBufs), (c / kBufs) & 1, flag, limit);
            float x[16];  // a column of a diagonal block's inverse
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float acc0 = i == col ? 1.f : 0.f, acc1 = 0.f;
#pragma unroll
                for (int j = 0; j < i; j += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(d + diag_at(i, j));
                    acc0 = fmaf(-a.x, x[j], acc0);
                    if (j + 1 < i) acc1 = fmaf(-a.y, x[j + 1], acc1);
                    if (j + 2 < i) acc0 = fmaf(-a.z, x[j + 2], acc0);
                    if (j + 3 < i) acc1 = fmaf(-a.w, x[j + 3], acc1);
                }
                x[i] = acc0 + acc1;
            }
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                uint32_t hi, lo;
                split2(f2(x[i], x[i + 1]), hi, lo);
                const uint32_t off0 = sw128_off(16 * blk + i, 16 * blk + col), off1 = sw128_off(16 * blk + i + 1, 16 * blk + col);
                *reinterpret_cast<uint16_t *>(tp + off0) = static_cast<uint16_t>(hi);
                *reinterpret_cast<uint16_t *>(tp + off1) = static_cast<uint16_t>(hi >> 16);
                *reinterpret_cast<uint16_t *>(tp + kTile + off0) = static_cast<uint16_t>(lo);
                *reinterpret_cast<uint16_t *>(tp + kTile + off1) = static_cast<uint16_t>(lo >> 16);
            }
            const uint32_t t_hi = smem_addr(tp), a_hi = sbase + M::oA + (c % kBufs) * kTile;
            __syncwarp();
            off_diagonal<16>(t_hi, t_hi + kTile, a_hi, a_hi + kTile / 2, 32 * w, 0, 16 * w, 32, lane);
            bar_sync_named(5 + (c & 1), 64);
            off_diagonal<32>(t_hi, t_hi + kTile, a_hi, a_hi + kTile / 2, 0, 16 * w, 0, 0, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(prep_ready + 8 * (c % kBufs)), mbar_arrive(a_free + 8 * (c % kBufs));
        }
    } else {
        // ----------------------------------------------------- the scalars
        const int t = 16 * (warp - kScalWarp) + lane;
        const int h = head();
        float next_g = 0.f, next_beta = 0.f;
        auto fetch = [&](int c) {
            const bool in = c * kL + t < len;
            const long long row = static_cast<long long>(t0) + c * kL + t;
            next_g = in ? __ldg(p.in.g + row * p.in.g_stride + h) : 0.f;
            next_beta = in ? __ldg(p.in.beta + row * p.in.beta_stride + h) : 0.f;
        };
        fetch(0);
        for (int c = 0; c < n_chunks; ++c) {
            const int n = min(kL, len - c * kL);
            const float gv = next_g, beta = next_beta;
            fetch(c + 1);
            uint8_t *kq = base + M::oKQ + (c % kStagesKQ) * M::kKQ;
            float *sc = scal(c);
            // log2 decay as a pair, then its running sum over the chunk
            constexpr float kLog2e = 1.4426950408889634f;
            constexpr float kLog2eLo = static_cast<float>(1.4426950408889634074 - static_cast<double>(kLog2e));
            float gh = __fmul_rn(gv, kLog2e);
            float gl = fmaf(gv, kLog2eLo, fmaf(gv, kLog2e, -gh));
            if (gh < -160.f) gh = -160.f, gl = 0.f;  // -inf too; NaN stays
#pragma unroll 1
            for (int d = 1; d < 32; d <<= 1) {
                const float x = __shfl_up_sync(0xffffffffu, gh, d), y = __shfl_up_sync(0xffffffffu, gl, d);
                if (lane >= d) pair_add(gh, gl, x, y);
            }
            // the lengths of row t of K and of Q
            wait<true>(full_kq + 8 * (c % kStagesKQ), (c / kStagesKQ) & 1, flag, limit);
            float k0 = 0.f, k1 = 0.f, q0 = 0.f, q1 = 0.f;
#pragma unroll 1
            for (int hh = 0; hh < DK / 64; ++hh) {
                const uint8_t *tile = kq + hh * 2 * kTile;
#pragma unroll 4
                for (int j = 0; j < 8; ++j) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(tile + sw128_off(t, 8 * j));
                    const uint4 w = *reinterpret_cast<const uint4 *>(tile + kTile + sw128_off(t, 8 * j));
                    const uint32_t us[4] = {u.x, u.y, u.z, u.w}, ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        add_squares(us[e], k0, k1);
                        add_squares(ws[e], q0, q1);
                    }
                }
            }
            float nk = p.in.eps > 0.f ? rsqrtf(k0 + k1 + p.in.eps) : 1.f;
            const float nq = p.in.scale * (p.in.eps > 0.f ? rsqrtf(q0 + q1 + p.in.eps) : 1.f);
            if (t >= n) {  // whatever lies past the sequence must not meet E's zeros as NaN
                nk = 0.f;
#pragma unroll 1
                for (int hh = 0; hh < DK / 64; ++hh)
#pragma unroll 1
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4 *>(kq + hh * 2 * kTile + sw128_off(t, 8 * j)) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            // the running sum across the two warps, by way of the table of -G
            if (t == 31) sc[kGh * kL + 31] = -gh, sc[kGl * kL + 31] = -gl;
            bar_sync_named(11, 64);
            if (warp != kScalWarp) pair_add(gh, gl, -sc[kGh * kL + 31], -sc[kGl * kL + 31]);
            if (t != 31) sc[kGh * kL + t] = -gh, sc[kGl * kL + t] = -gl;
            bar_sync_named(11, 64);
            constexpr float kLn2 = 0.69314718f;
            const float gamma = ex2_approx(gh) * fmaf(gl, kLn2, 1.f);
            sc[kCx * kL + t] = -nk * gamma;
            sc[kCe * kL + t] = beta * nk * ex2_approx((-sc[kGh * kL + 63] - gh) + (-sc[kGl * kL + 63] - gl));
            sc[kCo * kL + t] = nq * gamma;
            sc[kNk * kL + t] = beta * nk;
            sc[kRowA * kL + t] = nk;
            sc[kRowP * kL + t] = nq;
            if (t == 63) sc[kScalRows * kL] = gamma;
            __syncwarp();
            if (lane == 0) mbar_arrive(scal_ready + 8 * (c % kScal));
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (TRANS && tid == 32) *gave_up = *flag;
    if (!TRANS && *redo && !*flag) {
        run_by_token<DK, DV>(p, marked, head(), t0, len, ck0, from, state_off, from_bf16, PIECES || to_pool ? to : nullptr, to_off,
                             to_pool && p.lv.state_bf16);
        __syncthreads();
    }
    if (PIECES && tid == 32 && !to_pool && !*flag) {  // the state that all chain warps wrote
        __threadfence();
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(sg.done + held[1]) : "memory");
    }
    if (warp == 0) {
        tc_fence_after();
        if (tid == 0 && *flag) flag_status(p.lv.status, WKV7_DEV_WAIT_TIMEOUT);
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ host side
// [tokens][heads][size] bf16 with rows `stride` elements apart; one box = 64 tokens x
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

// The states at the segments' starts: S_{j+1} = S_j Phi_j + Psi_j, written over Psi_j.  One
// CTA takes 16 value rows of one (sequence, head) through all segments; four warps of four
// rows, four columns a lane, Phi double buffered through shared memory.  Bound by shared
// memory: each warp reads all of Phi (about 1.2 us a segment at dk = 128).
constexpr int kJoinRows = 16, kJoinThreads = 128;

template <int DK>
__global__ void __launch_bounds__(kJoinThreads) gdn_join_kernel(const GdnRunArgs p, const Segments sg) {
    extern __shared__ __align__(16) uint8_t join_smem[];
    float *phi = reinterpret_cast<float *>(join_smem);  // [2][DK][DK]
    float *st = phi + 2 * DK * DK;                      // [kJoinRows][DK]
    pdl_prologue();
    const int seq = blockIdx.z, h = blockIdx.y, row0 = blockIdx.x * kJoinRows;
    const int slot = __ldg(p.slot_ids + seq);
    const int t0 = __ldg(p.cu_seqlens + seq), t1 = __ldg(p.cu_seqlens + seq + 1);
    if (slot < 0 || slot >= p.lv.n_slots || t0 < 0 || t1 <= t0 || t1 > p.total_tokens || t1 - t0 > p.max_seqlen) return;
    const int joins = (t1 - t0 - 1) / sg.tokens;  // segments but the last
    if (joins == 0) return;
    const size_t unit = static_cast<size_t>(seq) * p.lv.hv + h;
    int bad = 0;
    for (int e = threadIdx.x; e < 2 * joins; e += kJoinThreads) bad |= sg.gave_up[unit * (sg.n - 1) * 2 + e];
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0 && row0 == 0) sg.lost[unit] = bad;
    if (bad) return;
    const float *phis = sg.phi + unit * (sg.n - 1) * DK * DK;
    float *psis = sg.psi + unit * sg.n * p.lv.dv * DK + static_cast<size_t>(row0) * DK;
    auto fetch = [&](int j) {
        const float *src = phis + static_cast<size_t>(j) * DK * DK;
        const uint32_t dst = smem_addr(phi + (j & 1) * DK * DK);
        for (int e = threadIdx.x * 4; e < DK * DK; e += kJoinThreads * 4)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 4 * e), "l"(src + e) : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(0);
    const size_t s_off = static_cast<size_t>(slot) * p.lv.slot_stride + p.lv.layer_off +
                         (static_cast<size_t>(h) * p.lv.dv + row0) * DK;
    for (int e = threadIdx.x * 4; e < kJoinRows * DK; e += kJoinThreads * 4) {
        const float4 x = p.lv.state_bf16 ? load_state4<true>(p.lv.states, s_off + e) : load_state4<false>(p.lv.states, s_off + e);
        *reinterpret_cast<float4 *>(st + e) = x;
        *reinterpret_cast<float4 *>(psis + e) = x;
    }
    const int lane = threadIdx.x & 31;
    const int r0 = 4 * (threadIdx.x >> 5) + (DK == 64 ? 2 * (lane >> 4) : 0);  // DK = 64: two rows a half-warp
    const int c = 4 * (DK == 64 ? (lane & 15) : lane);
    constexpr int R = DK == 64 ? 2 : 4;
    for (int j = 0; j < joins; ++j) {
        if (j + 1 < joins) {
            fetch(j + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        float *psi = psis + static_cast<size_t>(j + 1) * p.lv.dv * DK;
        float4 acc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = *reinterpret_cast<const float4 *>(psi + (r0 + r) * DK + c);
        __syncthreads();  // Phi_j and the state rows are there
        const float *f = phi + (j & 1) * DK * DK + c;
#pragma unroll 4
        for (int k = 0; k < DK; k += 4) {
            float4 s[R], y[4];
#pragma unroll
            for (int r = 0; r < R; ++r) s[r] = *reinterpret_cast<const float4 *>(st + (r0 + r) * DK + k);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = *reinterpret_cast<const float4 *>(f + (k + e) * DK);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float sr[4] = {s[r].x, s[r].y, s[r].z, s[r].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[r].x = fmaf(sr[e], y[e].x, acc[r].x);
                    acc[r].y = fmaf(sr[e], y[e].y, acc[r].y);
                    acc[r].z = fmaf(sr[e], y[e].z, acc[r].z);
                    acc[r].w = fmaf(sr[e], y[e].w, acc[r].w);
                }
            }
        }
        __syncthreads();  // the state rows and this half of Phi's buffer are read
#pragma unroll
        for (int r = 0; r < R; ++r) {
            *reinterpret_cast<float4 *>(st + (r0 + r) * DK + c) = acc[r];
            *reinterpret_cast<float4 *>(psi + (r0 + r) * DK + c) = acc[r];
        }
    }
}

template <int DK, int DV, bool OF32, Mode MODE>
cudaError_t launch_chunks(const GdnRunArgs &a, const Segments &sg, const Maps &maps, dim3 grid, cudaStream_t s) {
    constexpr int bytes = static_cast<int>(Smem<DK, DV, OF32>::kBytes) + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
    auto kernel = gdn_chunk_kernel<DK, DV, OF32, MODE>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return e != cudaSuccess ? e : launch_pdl(kernel, grid, dim3(kThreads), bytes, s, a, sg, maps);
}

__global__ void clear_kernel(unsigned *x, long long n) {
    pdl_prologue();
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < n) x[i] = 0;
}

template <int DK, int DV, bool OF32>
cudaError_t chunk_as(const GdnRunArgs &a, const GdnSplit &split, cudaStream_t s, int *launches) {
    Maps maps;
    if (!encode(&maps.q, a.in.q, DK, a.lv.hk, a.total_tokens, a.in.q_stride) ||
        !encode(&maps.k, a.in.k, DK, a.lv.hk, a.total_tokens, a.in.k_stride) ||
        !encode(&maps.v, a.in.v, DV, a.lv.hv, a.total_tokens, a.in.v_stride))
        return cudaErrorInvalidValue;
    const unsigned n = static_cast<unsigned>(a.n), heads = static_cast<unsigned>(a.lv.hv);
    Segments sg{};
    if (split.pieces) {
        const size_t units = static_cast<size_t>(n) * heads;
        sg.from1 = split.from1;
        sg.from2 = split.from2;
        sg.carry = static_cast<float *>(a.workspace);
        sg.done = reinterpret_cast<unsigned *>(sg.carry + units * DV * DK);
        const cudaError_t e = launch_pdl(clear_kernel, dim3(static_cast<unsigned>((units + 255) / 256)), dim3(256), 0, s, sg.done,
                                         static_cast<long long>(units));
        if (e != cudaSuccess) return e;
        *launches += 2;
        return launch_chunks<DK, DV, OF32, kPiece>(a, sg, maps, dim3(heads, n, 3), s);
    }
    if (split.segments < 2) {
        ++*launches;
        return launch_chunks<DK, DV, OF32, kWhole>(a, sg, maps, dim3(heads, n < 65535u ? n : 65535u, (n + 65534u) / 65535u), s);
    }
    sg.tokens = split.chunks * kL;
    sg.n = split.segments;
    sg.phi = static_cast<float *>(a.workspace);
    const size_t units = static_cast<size_t>(n) * heads;
    sg.psi = sg.phi + units * (sg.n - 1) * DK * DK;
    sg.gave_up = reinterpret_cast<int *>(sg.psi + units * sg.n * DV * DK);
    sg.lost = sg.gave_up + units * (sg.n - 1) * 2;
    const unsigned z = static_cast<unsigned>(sg.n - 1);
    cudaError_t e;
    if constexpr (DK == DV) {
        e = launch_chunks<DK, DV, false, kTransfer>(a, sg, maps, dim3(heads, n, 2 * z), s);
        ++*launches;
    } else {
        sg.kinds = 1;
        e = launch_chunks<DK, DV, false, kTransfer>(a, sg, maps, dim3(heads, n, z), s);
        ++*launches;
        if (e != cudaSuccess) return e;
        sg.kinds = 2;
        e = launch_chunks<DK, DK, false, kTransfer>(a, sg, maps, dim3(heads, n, z), s);
        ++*launches;
    }
    if (e != cudaSuccess) return e;
    constexpr int bytes = (2 * DK * DK + kJoinRows * DK) * 4;
    e = cudaFuncSetAttribute(gdn_join_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    e = launch_pdl(gdn_join_kernel<DK>, dim3(DV / kJoinRows, heads, n), dim3(kJoinThreads), bytes, s, a, sg);
    ++*launches;
    if (e != cudaSuccess) return e;
    ++*launches;
    return launch_chunks<DK, DV, OF32, kWhole>(a, sg, maps, dim3(heads, n, z + 1), s);
}

}  // namespace

bool gdn_chunk_takes(const GdnRunArgs &a) {
    return a.in.bf16 && a.cu_seqlens && a.total_tokens > 0 && a.in.q_stride > 0 && a.in.k_stride > 0 && a.in.v_stride > 0;
}

// One CTA runs on each of the 152 SMs.  Measured, us: a chunk of heads of 128 4.2, of 128 x 64 4.2, of 64
// x 128 3.7 (taken for 4.2 here), of 64 3.4 to 3.6, without outputs 5/6 of that, a CTA's start and end 8 to
// 11, a join step 1.3.
constexpr double kStartUs = 11, kJoinUs = 1.3;

// Units of about equal length that fill some rounds of the SMs but not the last leave SMs idle
// in it.  A unit is then taken in three pieces of 5/8, 2/8 and 1/8 of the longest sequence, all
// units' first pieces first: the SMs that the last round of long pieces leaves free take short
// ones.  Two more starts a unit have to be less than what is idle otherwise.  Whole and in
// pieces, us: 256 units of 64 chunks of heads of 128 535 and 505, 192 527 and 448, 160 of 17 148
// and 141, 320 of 32 397 and 345; heads of 64, 192 of 64 437 and 374, 160 of 64 385 and 338.  Left whole:
// 256 of 32 277, heads of 64, 160 of 17 113 (in pieces 2 to 4% more when the rule was chosen).
void plan_pieces(GdnSplit &split, double units_per_sm, int chunks, double chunk_us) {
    if (chunks < 16) return;
    const int b1 = (5 * chunks + 7) / 8, b2 = (7 * chunks + 7) / 8;
    const double whole = std::ceil(units_per_sm) * (kStartUs + chunk_us * chunks);
    const double packed = std::max(chunk_us * chunks * (units_per_sm + 0.0625), chunk_us * (b1 + chunks)) +
                          3 * kStartUs * units_per_sm + 3;
    if (packed > 0.95 * whole) return;
    split.pieces = 3;
    split.from1 = b1;
    split.from2 = b2;
}

// How to cut the sequences.  Where units fill the SMs, whole or in pieces; else the number of
// segments that gives the shortest estimate, if that promises a fifth less than the uncut time.
// Uncut and cut, us: 1 x 16,383 tokens x 8 heads of 128 977 and 225; 1 x 4,096 x 8 250 and 93,
// x 32 255 and 197; 4 x 2,048 x 8 130 and 111; 1 x 8,000 x 4 heads of 64 367 and 85.
GdnSplit gdn_plan_split(int n_seqs, int heads, int max_seqlen, int dk, int dv) {
    GdnSplit best{};
    const long long units = static_cast<long long>(n_seqs) * heads;
    const int chunks = (max_seqlen + kL - 1) / kL;
    const double chunk_us = dk * dv <= 64 * 64 ? 3.4 : 4.2;
    if (units > 152) {
        if (n_seqs <= 65535) plan_pieces(best, static_cast<double>(units) / 152, chunks, chunk_us);
        return best;
    }
    if (units <= 0 || units == 152 || chunks < 8) return best;
    auto rounds = [](long long ctas) { return static_cast<double>((ctas + 151) / 152); };
    double least = 0.8 * (kStartUs + chunk_us * chunks);
    for (int n = 2; n <= 64 && n * 4 <= chunks; ++n) {
        const int per = (chunks + n - 1) / n, used = (chunks + per - 1) / per;
        if (used != n) continue;
        const double t = rounds(units * (n - 1) * 2) * (kStartUs + chunk_us * 5 / 6 * per) + 6 + kJoinUs * (n - 1) +
                         rounds(units * n) * (kStartUs + chunk_us * per);
        if (t < least) {
            least = t;
            best.segments = n;
            best.chunks = per;
        }
    }
    return best;
}

size_t gdn_split_bytes(const GdnSplit &split, long long units, int dk, int dv) {
    const size_t n = static_cast<size_t>(split.segments);
    if (split.pieces) return static_cast<size_t>(units) * (static_cast<size_t>(dk) * dv * sizeof(float) + sizeof(int));
    if (split.segments < 2) return 0;
    const size_t words = static_cast<size_t>(units) * (2 * (n - 1) + 1);
    return static_cast<size_t>(units) * dk * ((n - 1) * dk + n * dv) * sizeof(float) + (words * sizeof(int) + 15) / 16 * 16;
}

cudaError_t launch_gdn_chunk(const GdnRunArgs &a, cudaStream_t s, int *launches) {
    GdnSplit split = gdn_plan_split(a.n, a.lv.hv, a.max_seqlen, a.lv.dk, a.lv.dv);
    // a checkpointed call has no segments: what a checkpoint resumes repeats this call's path
    // (pieces change no bit)
    if (a.cu_ckpt && split.segments) split = GdnSplit{};
    if (!a.workspace || a.workspace_bytes < gdn_split_bytes(split, static_cast<long long>(a.n) * a.lv.hv, a.lv.dk, a.lv.dv))
        split = GdnSplit{};
    cudaError_t (*const as[8])(const GdnRunArgs &, const GdnSplit &, cudaStream_t, int *) = {
        chunk_as<64, 64, false>,  chunk_as<64, 64, true>,  chunk_as<64, 128, false>,  chunk_as<64, 128, true>,
        chunk_as<128, 64, false>, chunk_as<128, 64, true>, chunk_as<128, 128, false>, chunk_as<128, 128, true>};
    const cudaError_t e = as[(a.lv.dk == 128 ? 4 : 0) | (a.lv.dv == 128 ? 2 : 0) | (a.in.o_bf16 ? 0 : 1)](a, split, s, launches);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace wkv7
