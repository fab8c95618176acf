// The gated delta rule over whole sequences, by chunks of 64 tokens on the tcgen05
// tensor cores.
//
// Per value head, S [dv][dk] (i value, j key), a token does
//     S <- exp(g) S;  e = beta (v - S k);  S <- S + e k^T;  o = scale S q.
// Over a chunk from state S0, with G_t the sum of the log decays up to token t and
// D_ts = exp(G_t - G_s), unrolling gives for the columns e_t
//     (I + A) E^T = diag(beta) (V - diag(exp G) K S0^T),   A_ts = beta_t D_ts <k_t, k_s>, s < t
//     O   = scale (diag(exp G) Q S0^T + P E^T),            P_ts = D_ts <q_t, k_s>, s <= t
//     S_L = exp(G_L) S0 + E diag(exp(G_L - G)) K
// All factors are exp of differences of G with s <= t, so at most 1: no decay is
// too strong.  G is kept as a pair of floats, so that a difference stays exact
// after a token that empties the state (g is taken as at least -160 log2 e; 2^-160
// is 0 in float32).
//
// Precision.  q, k and v are bf16 and go to the tensor cores as they were loaded:
// their lengths, decays, beta and scale are float32 factors on the accumulators.
// The computed operands (S0, the right-hand sides, E, T = (I + A)^-1 and P) are
// split into two bf16 parts, 16 bits; a product of two split operands leaves out
// only lo x lo (2^-18).  States stay float32 in tensor memory from chunk to chunk.
//
// One CTA owns one (sequence, value head) and walks its chunks.  Two pipelines
// share it.  "Prep" (warps 0-3) does what does not depend on the state, a chunk
// or so ahead: lengths and decays, the products K K^T and Q K^T, T by two 32 x 32
// triangular inverses and one off-diagonal block in float32, and the operand tiles
// of T and P.  The "chain" (warps 4-11) is the recurrence proper:
//     X  = S0 [K; Q]^T           M = dv, N = 128, K = dk, S0 from tensor memory
//     RHS = beta v - (beta exp(G) / |k|) X_K                      (CUDA cores)
//     E  = RHS T^T               M = dv, N = 64, K = 64, RHS from tensor memory
//     S += E' K                  M = dv, N = dk, K = 64, E' = E diag(..) from tensor memory
//     O  = E P^T                 M = dv, N = 64, K = 64
// Value rows sit in the accumulator's lanes throughout, so what one product leaves
// is the next one's A operand in the same lanes, written straight back to tensor
// memory; only T and P pass through shared memory.  Warp 12 issues the chain's
// MMAs, warp 13 the TMA loads (three chunks of k and q, two of v in flight), warp 14
// the prep MMAs.  All waits are bounded.
//
// Bound by the chain's latency: each chunk is four dependent products with a
// readback between them.
#include "device_common.cuh"
#include "gdn_internal.h"
#include "sm100_ptx.cuh"
#include "wkv7_internal.h"

namespace wkv7 {
namespace {

using namespace sm100;

constexpr int kL = 64;
constexpr int kThreads = 480;
constexpr int kPrepWarps = 4, kChainWarps = 8;
constexpr int kStagesKQ = 3, kBufs = 2, kScal = 4;
constexpr int kPitch = 68;  // floats per row of the float32 64 x 64 scratch (16-byte rows, no bank conflicts)

// Tensor-memory columns (512): S float32; its bf16 parts; X = [X_K | X_Q], whose
// halves become E's accumulator (then E's operand) and O's; RHS's operand (then
// E''s); prep's [K; Q] K^T.  A bf16 operand holds K elements 2c, 2c + 1 in column c.
constexpr uint32_t kColS = 0, kColSHi = 128, kColSLo = 192, kColX = 256, kColXQ = 320, kColR = 384, kColKKQ = 448;

struct Maps {
    CUtensorMap q, k, v;
};

// Shared memory, from the first 1024-byte boundary: tiles, then the small items.
constexpr uint32_t kTile = 8192;  // 64 rows of 128 bytes, 128-byte swizzle
// OF32: float32 outputs.  E P^T then keeps P in three parts and adds lo x lo: with
// keys that hardly differ the e_t telescope, |sum P e| is far below sum |P e|, and
// two parts left errors of 5e-5 of the largest output (200 tokens of such keys;
// three: 2.6e-5).  A bf16 output rounds at 2e-3, two parts are enough.
template <int DK, int DV, bool OF32>
struct Smem {
    static constexpr int kStagesV = OF32 ? 1 : 2;      // the third part of P takes the second one's place
    static constexpr uint32_t kTP = (OF32 ? 5 : 4) * kTile;
    static constexpr uint32_t kKQ = DK / 64 * 2 * kTile;  // per stage: for each 64 of dk, K rows then Q rows
    static constexpr uint32_t kV = DV / 64 * kTile;
    static constexpr uint32_t oKQ = 0;
    static constexpr uint32_t oV = oKQ + kStagesKQ * kKQ;
    static constexpr uint32_t oTP = oV + kStagesV * kV;  // per buffer: T hi, T lo, P hi, P lo(, P's third part): rows t, 64 columns s
    static constexpr uint32_t oA = oTP + kBufs * kTP;
    static constexpr uint32_t oScal = oA + kL * kPitch * 4;  // per buffer: cx, beta, ce, co [64] and gl
    static constexpr uint32_t kScalBytes = 4 * kL * 4 + 16;
    static constexpr uint32_t oPrep = oScal + kScal * kScalBytes;  // nk, G hi, G lo [64], warp total
    static constexpr uint32_t oBar = oPrep + 3 * kL * 4 + 16;
    static constexpr uint32_t kBars = 2 * kStagesKQ + 2 * kStagesV + 2 + kScal + 2 * kBufs + 8 + 2;
    static constexpr uint32_t oHold = oBar + kBars * 8;
    static constexpr uint32_t kBytes = oHold + 16;
};

__device__ __forceinline__ float ex2_approx(float x) {  // 2 ulp, 2^x for x <= -149 is 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two floats as bf16 pairs: the rounded values and what they leave.
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16_rn(a, b);
    lo = pack_bf16_rn(a - bf16_lo(hi), b - bf16_hi(hi));
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A wait that ends: with the phase, when another role has given up, or after the limit.
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, volatile int *flag, long long limit) {
    if (mbar_try_wait(bar, parity)) return;
    const long long t0 = clock64();
    while (!mbar_try_wait_sleep(bar, parity, 1000u)) {
        if (*flag) return;
        if (clock64() - t0 > limit) {
            *flag = 1;
            return;
        }
    }
}

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

template <int DK, int DV, bool OF32>
__global__ void __launch_bounds__(512, 1) gdn_chunk_kernel(const GdnRunArgs p, const __grid_constant__ Maps maps) {
    using M = Smem<DK, DV, OF32>;
    constexpr int kStagesV = M::kStagesV;
    extern __shared__ uint8_t smem_raw[];
    pdl_prologue();
    const int h = blockIdx.x, seq = blockIdx.y + blockIdx.z * 65535;
    if (seq >= p.n) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slot = __ldg(p.slot_ids + seq);
    const int t0 = __ldg(p.cu_seqlens + seq), t1 = __ldg(p.cu_seqlens + seq + 1);
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
    const int len = t1 - t0;
    if (len == 0) return;
    const int n_chunks = (len + kL - 1) / kL;
    const int hk = h / (p.lv.hv / p.lv.hk);

    uint8_t *base = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(base);
    volatile int *flag = reinterpret_cast<volatile int *>(base + M::oHold + 4);
    uint32_t nbar = sbase + M::oBar;
    auto bars = [&nbar](int n) { const uint32_t b = nbar; nbar += 8 * n; return b; };
    const uint32_t full_kq = bars(kStagesKQ), kq_empty = bars(kStagesKQ), full_v = bars(kStagesV), v_empty = bars(kStagesV);
    const uint32_t kkq_full = bars(1), kkq_free = bars(1), scal_ready = bars(kScal), prep_ready = bars(kBufs);
    const uint32_t buf_free = bars(kBufs), bar_x = bars(1), bar_rhs = bars(1), bar_e = bars(1), bar_ep = bars(1);
    const uint32_t bar_eo = bars(1), bar_s = bars(1), bar_o = bars(1), s_ready = bars(1), drain = bars(2);
    const long long limit = p.wait_cycles;

    if (warp == 0) tmem_alloc(sbase + M::oHold, 512);
    if (tid == 32) {
        for (int i = 0; i < kStagesKQ; ++i) mbar_init(full_kq + 8 * i, 1), mbar_init(kq_empty + 8 * i, 1);
        for (int i = 0; i < kStagesV; ++i) mbar_init(full_v + 8 * i, 1), mbar_init(v_empty + 8 * i, kChainWarps);
        for (int i = 0; i < kScal; ++i) mbar_init(scal_ready + 8 * i, kPrepWarps);
        for (int i = 0; i < kBufs; ++i) mbar_init(prep_ready + 8 * i, kPrepWarps), mbar_init(buf_free + 8 * i, kChainWarps);
        mbar_init(kkq_full, 1), mbar_init(kkq_free, kPrepWarps);
        mbar_init(bar_x, 1), mbar_init(bar_e, 1), mbar_init(bar_s, 1), mbar_init(bar_o, 1);
        mbar_init(bar_rhs, kChainWarps), mbar_init(bar_ep, kChainWarps), mbar_init(bar_eo, kChainWarps);
        mbar_init(s_ready, kChainWarps);
        mbar_init(drain, 1), mbar_init(drain + 8, 1);
        fence_mbar_init();
        *flag = 0;
    }
    // T and P are lower triangular: their upper right 32 x 32 blocks are zeros for good
    for (int e = tid; e < static_cast<int>(kBufs * M::kTP / kTile) * 32 * 4; e += kThreads) {
        const int tile = e / 128, row = (e / 4) % 32, c = 32 + (e % 4) * 8;
        *reinterpret_cast<uint4 *>(base + M::oTP + tile * kTile + sw128_off(row, c)) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(base + M::oHold);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    auto scal = [base](int c) { return reinterpret_cast<float *>(base + M::oScal + (c % kScal) * M::kScalBytes); };

    if (warp < kPrepWarps) {
        // ------------------------------------------------------------- prep
        float *A = reinterpret_cast<float *>(base + M::oA);
        float *s_nk = reinterpret_cast<float *>(base + M::oPrep), *s_gh = s_nk + kL, *s_gl = s_gh + kL, *s_tot = s_gl + kL;
        const int m = tid, t = m & 63;
        const bool is_q = m >= 64;
        const float *gate = is_q ? p.in.beta + h : p.in.g + h;
        const long long gate_stride = is_q ? p.in.beta_stride : p.in.g_stride;
        float next_gate = t < len ? __ldg(gate + (t0 + t) * gate_stride) : 0.f;
        // (after a wait gave up the loops below run on, on whatever they find: the warps of
        // a named barrier must all come to it, and no wait holds them any more)
        for (int c = 0; c < n_chunks; ++c) {
            const int n = min(kL, len - c * kL);
            const float gv = next_gate;
            const int ahead = (c + 1) * kL + t;
            next_gate = ahead < len ? __ldg(gate + (static_cast<long long>(t0) + ahead) * gate_stride) : 0.f;
            uint8_t *kq = base + M::oKQ + (c % kStagesKQ) * M::kKQ;
            float *sc = scal(c);
            wait(full_kq + 8 * (c % kStagesKQ), (c / kStagesKQ) & 1, flag, limit);
            // this row's length
            float ss = 0.f;
#pragma unroll
            for (int hh = 0; hh < DK / 64; ++hh) {
                const uint8_t *tile = kq + hh * 2 * kTile + (is_q ? kTile : 0);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(tile + sw128_off(t, 8 * j));
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        ss = fmaf(bf16_lo(w[e]), bf16_lo(w[e]), ss);
                        ss = fmaf(bf16_hi(w[e]), bf16_hi(w[e]), ss);
                    }
                }
            }
            float inv = p.in.eps > 0.f ? rsqrtf(ss + p.in.eps) : 1.f;
            if (t >= n) inv = 0.f;
            float gh = 0.f, gl = 0.f;
            if (!is_q) {
                if (t >= n) {  // whatever lies past the sequence must not meet E's zeros as NaN
#pragma unroll
                    for (int hh = 0; hh < DK / 64; ++hh)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint4 *>(kq + hh * 2 * kTile + sw128_off(t, 8 * j)) = make_uint4(0, 0, 0, 0);
                }
                // log2 decay as a pair, then its running sum over the chunk
                constexpr float kLog2e = 1.4426950408889634f;
                constexpr float kLog2eLo = static_cast<float>(1.4426950408889634074 - static_cast<double>(kLog2e));
                gh = __fmul_rn(gv, kLog2e);
                gl = fmaf(gv, kLog2eLo, fmaf(gv, kLog2e, -gh));
                if (gh < -160.f) gh = -160.f, gl = 0.f;  // -inf too; NaN stays
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const float x = __shfl_up_sync(0xffffffffu, gh, d), y = __shfl_up_sync(0xffffffffu, gl, d);
                    if (lane >= d) pair_add(gh, gl, x, y);
                }
                if (t == 31) s_tot[0] = gh, s_tot[1] = gl;
                s_nk[t] = inv;
            } else {
                sc[kL + t] = t < n ? gv : 0.f;  // beta
            }
            bar_sync_named(5, 128);
            if (!is_q) {
                if (warp == 1) pair_add(gh, gl, s_tot[0], s_tot[1]);
                s_gh[t] = gh;
                s_gl[t] = gl;
            }
            bar_sync_named(5, 128);
            constexpr float kLn2 = 0.69314718f;
            gh = s_gh[t];
            gl = s_gl[t];
            const float gamma = ex2_approx(gh) * fmaf(gl, kLn2, 1.f);
            float row_c;  // this row's factor of its products with k
            if (!is_q) {
                const float beta = sc[kL + t];
                row_c = beta * inv;
                sc[t] = row_c * gamma;
                sc[2 * kL + t] = inv * ex2_approx((s_gh[63] - gh) + (s_gl[63] - gl));
                if (t == 63) sc[4 * kL] = gamma;
            } else {
                row_c = p.in.scale * inv;
                sc[3 * kL + t] = row_c * gamma;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(scal_ready + 8 * (c % kScal));

            // A (rows of K) and P (rows of Q) from the products with K
            uint8_t *tp = base + M::oTP + (c % kBufs) * M::kTP;
            wait(buf_free + 8 * (c % kBufs), ((c / kBufs) & 1) ^ 1, flag, limit);
            wait(kkq_full, c & 1, flag, limit);
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                if (b == 1 && (warp & 1) == 0) break;  // rows below 32 end at column 31
                float x[32];
                tmem_ld32(lane_base + kColKKQ + 32 * b, x);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const int s = 32 * b + j;
                    const float4 a = *reinterpret_cast<const float4 *>(s_gh + s);
                    const float4 l = *reinterpret_cast<const float4 *>(s_gl + s);
                    const float4 k = *reinterpret_cast<const float4 *>(s_nk + s);
                    const float as[4] = {a.x, a.y, a.z, a.w}, ls[4] = {l.x, l.y, l.z, l.w}, ks[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float f = row_c * ks[e] * ex2_approx((gh - as[e]) + (gl - ls[e]));
                        const bool keep = is_q ? s + e <= t : (s + e < t && t < n);
                        x[j + e] = keep ? f * x[j + e] : 0.f;
                    }
                }
                if (is_q) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        uint32_t hi[4], lo[4];
                        const uint32_t off = sw128_off(t, 32 * b + j);
#pragma unroll
                        for (int e = 0; e < 4; ++e) split2(x[j + 2 * e], x[j + 2 * e + 1], hi[e], lo[e]);
                        if constexpr (OF32) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = pack_bf16_rn((x[j + 2 * e] - bf16_lo(hi[e])) - bf16_lo(lo[e]),
                                                    (x[j + 2 * e + 1] - bf16_hi(hi[e])) - bf16_hi(lo[e]));
                            *reinterpret_cast<uint4 *>(tp + 4 * kTile + off) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        *reinterpret_cast<uint4 *>(tp + 2 * kTile + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4 *>(tp + 3 * kTile + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<float4 *>(A + t * kPitch + 32 * b + j) =
                            make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(kkq_free);
            bar_sync_named(5, 128);

            // T = (I + A)^-1: the two 32 x 32 diagonal blocks by forward substitution, a column a thread
            if (warp < 2) {
                const float *D = A + 32 * warp * kPitch + 32 * warp;
                float x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float acc0 = i == lane ? 1.f : 0.f, acc1 = 0.f;
#pragma unroll
                    for (int j = 0; j < i; j += 4) {
                        const float4 a = *reinterpret_cast<const float4 *>(D + i * kPitch + j);
                        acc0 = fmaf(-a.x, x[j], acc0);
                        if (j + 1 < i) acc1 = fmaf(-a.y, x[j + 1], acc1);
                        if (j + 2 < i) acc0 = fmaf(-a.z, x[j + 2], acc0);
                        if (j + 3 < i) acc1 = fmaf(-a.w, x[j + 3], acc1);
                    }
                    x[i] = acc0 + acc1;
                }
                __syncwarp();
                float *W = A + 32 * warp * kPitch + 32 * warp + lane;
#pragma unroll
                for (int i = 0; i < 32; ++i) W[i * kPitch] = x[i];
            }
            bar_sync_named(5, 128);
            // T21 = -T22 (A21 T11), A21 T11 by way of the unused upper right block
#pragma unroll
            for (int step = 0; step < 2; ++step) {
                const int r = m >> 2, cg = (m & 3) * 8;
                const float *left = A + (32 + r) * kPitch + 32 * step;
                const float *right = A + 32 * step + cg;
                float acc[8] = {};
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(left + j);
                    const float as[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 y = *reinterpret_cast<const float4 *>(right + (j + e) * kPitch);
                        const float4 z = *reinterpret_cast<const float4 *>(right + (j + e) * kPitch + 4);
                        acc[0] = fmaf(as[e], y.x, acc[0]); acc[1] = fmaf(as[e], y.y, acc[1]);
                        acc[2] = fmaf(as[e], y.z, acc[2]); acc[3] = fmaf(as[e], y.w, acc[3]);
                        acc[4] = fmaf(as[e], z.x, acc[4]); acc[5] = fmaf(as[e], z.y, acc[5]);
                        acc[6] = fmaf(as[e], z.z, acc[6]); acc[7] = fmaf(as[e], z.w, acc[7]);
                    }
                }
                const float sign = step == 0 ? 1.f : -1.f;
                float *out = step == 0 ? A + r * kPitch + 32 + cg : A + (32 + r) * kPitch + cg;
                *reinterpret_cast<float4 *>(out) = make_float4(sign * acc[0], sign * acc[1], sign * acc[2], sign * acc[3]);
                *reinterpret_cast<float4 *>(out + 4) = make_float4(sign * acc[4], sign * acc[5], sign * acc[6], sign * acc[7]);
                bar_sync_named(5, 128);
            }
            const int row = m >> 1, part = 32 * (m & 1);
            if (row >= 32 || part == 0) {
#pragma unroll
                for (int j = 0; j < 32; j += 8) {
                    const float4 y = *reinterpret_cast<const float4 *>(A + row * kPitch + part + j);
                    const float4 z = *reinterpret_cast<const float4 *>(A + row * kPitch + part + j + 4);
                    uint32_t hi[4], lo[4];
                    split2(y.x, y.y, hi[0], lo[0]);
                    split2(y.z, y.w, hi[1], lo[1]);
                    split2(z.x, z.y, hi[2], lo[2]);
                    split2(z.z, z.w, hi[3], lo[3]);
                    const uint32_t off = sw128_off(row, part + j);
                    *reinterpret_cast<uint4 *>(tp + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(tp + kTile + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(prep_ready + 8 * (c % kBufs));
        }
    } else if (warp < kPrepWarps + kChainWarps) {
        // ------------------------------------------------------------ chain
        const int half = (warp - kPrepWarps) >> 2;  // of each product's columns
        const int i = 32 * (warp & 3) + lane;       // value row
        const bool active = i < DV;                 // the same for a whole warp
        constexpr int kSCols = DK / 2;              // state columns of this thread
        const size_t head_off = p.lv.layer_off + (static_cast<size_t>(h) * DV + i) * DK + half * kSCols;
        const size_t s_off = static_cast<size_t>(slot) * p.lv.slot_stride + head_off;
        const bool sb = p.lv.state_bf16;

        // A state row part: float32 to tensor memory times the chunk's decay, and its bf16 parts.
        auto put_state = [&](const float (&s)[32], int b, float decay) {
            uint32_t hi[16], lo[16], f[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) split2(s[2 * e], s[2 * e + 1], hi[e], lo[e]);
            tmem_st16(lane_base + kColSHi + half * (kSCols / 2) + 16 * b, hi);
            tmem_st16(lane_base + kColSLo + half * (kSCols / 2) + 16 * b, lo);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e] = __float_as_uint(s[16 * g + e] * decay);
                tmem_st16(lane_base + kColS + half * kSCols + 32 * b + 16 * g, f);
            }
        };
        auto write_state = [&](float *dst, size_t off, const float (&s)[32]) {
            if (sb) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = pack_bf16_rn(s[2 * e], s[2 * e + 1]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(dst) + off)[e] =
                        make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    reinterpret_cast<float4 *>(dst + off)[e] =
                        make_float4(s[4 * e], s[4 * e + 1], s[4 * e + 2], s[4 * e + 3]);
            }
        };

        wait(scal_ready, 0, flag, limit);
        if (active) {
            const float decay = scal(0)[4 * kL];
#pragma unroll 1
            for (int b = 0; b < kSCols / 32; ++b) {
                float s[32];
                if (sb) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(p.lv.states) + s_off + 32 * b);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint4 u = src[e];
                        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int x = 0; x < 4; ++x) s[8 * e + 2 * x] = bf16_lo(w[x]), s[8 * e + 2 * x + 1] = bf16_hi(w[x]);
                    }
                } else {
                    const float4 *src = reinterpret_cast<const float4 *>(p.lv.states + s_off + 32 * b);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 u = src[e];
                        s[4 * e] = u.x, s[4 * e + 1] = u.y, s[4 * e + 2] = u.z, s[4 * e + 3] = u.w;
                    }
                }
                put_state(s, b, decay);
            }
            tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_ready);

        for (int c = 0; c < n_chunks; ++c) {
            const int n = min(kL, len - c * kL);
            const uint32_t ph = c & 1;
            const float *sc = scal(c);
            float xq[32];
            // RHS = beta v - cx X_K
            wait(bar_x, ph, flag, limit);
            wait(full_v + 8 * (c % kStagesV), (c / kStagesV) & 1, flag, limit);
            tc_fence_after();
            if (active) {
                float x[32];
                tmem_ld32(lane_base + kColX + 32 * half, x);
                tmem_ld32(lane_base + kColXQ + 32 * half, xq);
                const uint8_t *vt = base + M::oV + (c % kStagesV) * M::kV + (i >> 6) * kTile;
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(
                                               vt + sw128_off(32 * half + j, i & 63))) << 16);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 cx = *reinterpret_cast<const float4 *>(sc + 32 * half + j);
                    const float4 be = *reinterpret_cast<const float4 *>(sc + kL + 32 * half + j);
                    x[j] = fmaf(be.x, v[j], -cx.x * x[j]);
                    x[j + 1] = fmaf(be.y, v[j + 1], -cx.y * x[j + 1]);
                    x[j + 2] = fmaf(be.z, v[j + 2], -cx.z * x[j + 2]);
                    x[j + 3] = fmaf(be.w, v[j + 3], -cx.w * x[j + 3]);
                }
                if (n < kL) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (32 * half + j >= n) x[j] = 0.f;
                }
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) split2(x[2 * e], x[2 * e + 1], hi[e], lo[e]);
                tmem_st16(lane_base + kColR + 16 * half, hi);
                tmem_st16(lane_base + kColR + 32 + 16 * half, lo);
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_rhs), mbar_arrive(v_empty + 8 * (c % kStagesV));

            // E, and E' = E ce for the state
            wait(bar_e, ph, flag, limit);
            tc_fence_after();
            float e_[32];
            if (active) {
                tmem_ld32(lane_base + kColX + 32 * half, e_);
                tmem_ld_wait();
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float4 ce = *reinterpret_cast<const float4 *>(sc + 2 * kL + 32 * half + 2 * e);
                    split2(ce.x * e_[2 * e], ce.y * e_[2 * e + 1], hi[e], lo[e]);
                    split2(ce.z * e_[2 * e + 2], ce.w * e_[2 * e + 3], hi[e + 1], lo[e + 1]);
                }
                tmem_st16(lane_base + kColR + 16 * half, hi);
                tmem_st16(lane_base + kColR + 32 + 16 * half, lo);
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_ep);
            bar_sync_named(6 + (warp & 3), 64);  // both column halves of E are read: its columns take E's operand
            if (active) {
                tc_fence_after();
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) split2(e_[2 * e], e_[2 * e + 1], hi[e], lo[e]);
                tmem_st16(lane_base + kColX + 16 * half, hi);
                tmem_st16(lane_base + kColX + 32 + 16 * half, lo);
                tmem_st_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_eo);

            // the new state
            const bool last = c + 1 == n_chunks;
            int ck = -1;
            if (p.cu_ckpt && n == kL) {
                ck = __ldg(p.ckpt_ids + ck0 + c);
                if (ck < 0 || ck >= p.lv.n_snaps) {
                    if (tid == 32 * kPrepWarps) flag_status(p.lv.status, WKV7_DEV_BAD_SLOT);
                    ck = -1;
                }
            }
            if (!last) wait(scal_ready + 8 * ((c + 1) % kScal), ((c + 1) / kScal) & 1, flag, limit);
            wait(bar_s, ph, flag, limit);
            tc_fence_after();
            if (active) {
                const float decay = last ? 0.f : scal(c + 1)[4 * kL];
#pragma unroll 1
                for (int b = 0; b < kSCols / 32; ++b) {
                    float s[32];
                    tmem_ld32(lane_base + kColS + half * kSCols + 32 * b, s);
                    tmem_ld_wait();
                    if (sb && p.cu_ckpt && n == kL) {  // the carry goes on from what a checkpoint stores
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[e] = round_bf16(s[e]);
                    }
                    if (ck >= 0) write_state(p.lv.snaps, static_cast<size_t>(ck) * p.lv.slot_stride + head_off + 32 * b, s);
                    if (last) {
                        if (!*flag) write_state(p.lv.states, s_off + 32 * b, s);
                    } else {
                        put_state(s, b, decay);
                    }
                }
                tmem_st_wait();
            }
            // the outputs: O = co X_Q + E P^T
            wait(bar_o, ph, flag, limit);
            tc_fence_after();
            float o[32];
            if (active) {
                tmem_ld32(lane_base + kColXQ + 32 * half, o);
                tmem_ld_wait();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_ready);
            if (active) {
                const size_t step = static_cast<size_t>(p.lv.hv) * DV;
                const size_t at = (static_cast<size_t>(t0) + c * kL + 32 * half) * step + static_cast<size_t>(h) * DV + i;
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 co = *reinterpret_cast<const float4 *>(sc + 3 * kL + 32 * half + j);
                    o[j] = fmaf(co.x, xq[j], o[j]);
                    o[j + 1] = fmaf(co.y, xq[j + 1], o[j + 1]);
                    o[j + 2] = fmaf(co.z, xq[j + 2], o[j + 2]);
                    o[j + 3] = fmaf(co.w, xq[j + 3], o[j + 3]);
                }
                if constexpr (!OF32) {
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.in.o) + at;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (32 * half + j < n) dst[j * step] = __float2bfloat16_rn(o[j]);
                } else {
                    float *dst = static_cast<float *>(p.in.o) + at;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (32 * half + j < n) dst[j * step] = o[j];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(buf_free + 8 * (c % kBufs));
        }
    } else if (warp == 12) {
        // -------------------------------------------------- the chain's MMAs
        if (lane == 0) {
            for (int c = 0; c < n_chunks; ++c) {
                if (*flag) break;
                const uint32_t ph = c & 1;
                const uint32_t kq = sbase + M::oKQ + (c % kStagesKQ) * M::kKQ;
                const uint32_t tp = sbase + M::oTP + (c % kBufs) * M::kTP;
                wait(full_kq + 8 * (c % kStagesKQ), (c / kStagesKQ) & 1, flag, limit);
                wait(s_ready, ph, flag, limit);
                if (*flag) break;
                tc_fence_after();
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int hh = 0; hh < DK / 64; ++hh)
                        umma_ta_128xNx64(tmem + kColX, tmem + (part ? kColSLo : kColSHi) + 32 * hh, kq + hh * 2 * kTile, 128,
                                         part + hh > 0, false);
                umma_commit(bar_x);
                wait(prep_ready + 8 * (c % kBufs), (c / kBufs) & 1, flag, limit);
                wait(bar_rhs, ph, flag, limit);
                if (*flag) break;
                tc_fence_after();
                umma_ta_128xNx64(tmem + kColX, tmem + kColR, tp, 64, false, false);
                umma_ta_128xNx64(tmem + kColX, tmem + kColR + 32, tp, 64, true, false);
                umma_ta_128xNx64(tmem + kColX, tmem + kColR, tp + kTile, 64, true, false);
                umma_commit(bar_e);
                wait(bar_ep, ph, flag, limit);
                if (*flag) break;
                tc_fence_after();
                umma_ta_128xNx64(tmem + kColS, tmem + kColR, kq, DK, true, true, 2 * kTile);
                umma_ta_128xNx64(tmem + kColS, tmem + kColR + 32, kq, DK, true, true, 2 * kTile);
                umma_commit(bar_s);
                umma_commit(kq_empty + 8 * (c % kStagesKQ));
                wait(bar_eo, ph, flag, limit);
                if (*flag) break;
                tc_fence_after();
                umma_ta_128xNx64(tmem + kColXQ, tmem + kColX, tp + 2 * kTile, 64, false, false);
                umma_ta_128xNx64(tmem + kColXQ, tmem + kColX + 32, tp + 2 * kTile, 64, true, false);
                umma_ta_128xNx64(tmem + kColXQ, tmem + kColX, tp + 3 * kTile, 64, true, false);
                if constexpr (OF32) {
                    umma_ta_128xNx64(tmem + kColXQ, tmem + kColX + 32, tp + 3 * kTile, 64, true, false);
                    umma_ta_128xNx64(tmem + kColXQ, tmem + kColX, tp + 4 * kTile, 64, true, false);
                }
                umma_commit(bar_o);
            }
            if (*flag) {  // let what was issued end before the tensor memory goes
                umma_commit(drain);
                mbar_wait_bounded(drain, 0, limit);
            }
        }
    } else if (warp == 13) {
        // ------------------------------------------------------ input loads
        if (lane == 0) {
            int issued = 0;
            for (int c = 0; c < n_chunks; ++c) {
                const int sk = c % kStagesKQ, sv = c % kStagesV, at = t0 + c * kL;
                wait(kq_empty + 8 * sk, ((c / kStagesKQ) & 1) ^ 1, flag, limit);
                wait(v_empty + 8 * sv, ((c / kStagesV) & 1) ^ 1, flag, limit);
                if (*flag || p.test_skip_first_load) break;
                mbar_arrive_expect_tx(full_kq + 8 * sk, M::kKQ);
                const uint32_t kq = sbase + M::oKQ + sk * M::kKQ;
                for (int hh = 0; hh < DK / 64; ++hh) {
                    tma_load_3d(kq + hh * 2 * kTile, &maps.k, 64 * hh, hk, at, full_kq + 8 * sk);
                    tma_load_3d(kq + hh * 2 * kTile + kTile, &maps.q, 64 * hh, hk, at, full_kq + 8 * sk);
                }
                mbar_arrive_expect_tx(full_v + 8 * sv, M::kV);
                for (int hh = 0; hh < DV / 64; ++hh)
                    tma_load_3d(sbase + M::oV + sv * M::kV + hh * kTile, &maps.v, 64 * hh, h, at, full_v + 8 * sv);
                issued = c + 1;
            }
            if (*flag)  // let the copies in flight land
                for (int c = max(0, issued - kStagesKQ); c < issued; ++c) {
                    mbar_wait_bounded(full_kq + 8 * (c % kStagesKQ), (c / kStagesKQ) & 1, limit);
                    if (c >= issued - kStagesV) mbar_wait_bounded(full_v + 8 * (c % kStagesV), (c / kStagesV) & 1, limit);
                }
        }
    } else {
        // --------------------------------------------------- prep's products
        if (lane == 0) {
            for (int c = 0; c < n_chunks; ++c) {
                const uint32_t kq = sbase + M::oKQ + (c % kStagesKQ) * M::kKQ;
                wait(full_kq + 8 * (c % kStagesKQ), (c / kStagesKQ) & 1, flag, limit);
                wait(kkq_free, (c & 1) ^ 1, flag, limit);
                if (*flag) break;
                tc_fence_after();
#pragma unroll
                for (int hh = 0; hh < DK / 64; ++hh)
                    umma_128xNx64(tmem + kColKKQ, kq + hh * 2 * kTile, kq + hh * 2 * kTile, 64, hh > 0);
                umma_commit(kkq_full);
            }
            if (*flag) {
                umma_commit(drain + 8);
                mbar_wait_bounded(drain + 8, 0, limit);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        if (tid == 0 && *flag) flag_status(p.lv.status, WKV7_DEV_WAIT_TIMEOUT);
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = []() -> EncodeTiledFn {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

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

template <int DK, int DV, bool OF32>
cudaError_t chunk_as(const GdnRunArgs &a, cudaStream_t s) {
    Maps maps;
    if (!encode(&maps.q, a.in.q, DK, a.lv.hk, a.total_tokens, a.in.q_stride) ||
        !encode(&maps.k, a.in.k, DK, a.lv.hk, a.total_tokens, a.in.k_stride) ||
        !encode(&maps.v, a.in.v, DV, a.lv.hv, a.total_tokens, a.in.v_stride))
        return cudaErrorInvalidValue;
    constexpr int bytes = static_cast<int>(Smem<DK, DV, OF32>::kBytes) + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory of one CTA");
    cudaError_t e = cudaFuncSetAttribute(gdn_chunk_kernel<DK, DV, OF32>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const unsigned n = static_cast<unsigned>(a.n);
    const dim3 grid(static_cast<unsigned>(a.lv.hv), n < 65535u ? n : 65535u, (n + 65534u) / 65535u);
    return launch_pdl(gdn_chunk_kernel<DK, DV, OF32>, grid, dim3(kThreads), bytes, s, a, maps);
}

}  // namespace

bool gdn_chunk_takes(const GdnRunArgs &a) {
    return a.in.bf16 && a.cu_seqlens && a.total_tokens > 0 && a.in.q_stride > 0 && a.in.k_stride > 0 && a.in.v_stride > 0;
}

cudaError_t launch_gdn_chunk(const GdnRunArgs &a, cudaStream_t s, int *launches) {
    cudaError_t (*const as[8])(const GdnRunArgs &, cudaStream_t) = {
        chunk_as<64, 64, false>,  chunk_as<64, 64, true>,  chunk_as<64, 128, false>,  chunk_as<64, 128, true>,
        chunk_as<128, 64, false>, chunk_as<128, 64, true>, chunk_as<128, 128, false>, chunk_as<128, 128, true>};
    const cudaError_t e = as[(a.lv.dk == 128 ? 4 : 0) | (a.lv.dv == 128 ? 2 : 0) | (a.in.o_bf16 ? 0 : 1)](a, s);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace wkv7
