// The gated delta rule token by token: single-token decode over indirected state
// slots, and runs of tokens (multi-token decode with rollback states, prefill in
// float32).
//
// Per value head (S[i][j]: i value, j key) every token does
//     S <- exp(g) S;  e = beta (v - S k);  S <- S + e k^T;  o = scale S q.
// Row i of S needs only itself, k, q and v_i, so any set of rows is a unit of
// work: a warp holds kRows of them per lane group in registers, 16 bytes of a
// row per lane.  With the old row s both products come from one pass,
//     S k -> exp(g) (s k),    S' q = exp(g) (s q) + e (k q),
// so a token costs one round of shuffles (the sums of s k and s q for four rows
// scattered over the lanes: 9 shuffles for 32 lanes), not two in a row.  The
// lengths of q and k enter as factors on those sums.
//
// Decode is bound by HBM: a 128 x 128 float32 head moves 128 KiB for ~100 kFLOP.  256 slots
// of 32 such heads, 1.08 GB, take 153-158 us (6.8-7.0 TB/s, the copy rate); one slot 2.3 us,
// the launch and three dependent reads; 201 slots of 12 heads of 64 in bf16, 40 MB that stay in
// L2, 9.3 us.  A run with a state to keep after each token is bound by writing them: 48 slots x
// 5 tokens x 32 heads, 0.71 GB, 107 us (6.7 TB/s); without them by the shuffles and the inputs'
// staging (1 sequence of 24 tokens 14.7 us, of 128 66).
#include <type_traits>

#include "device_common.cuh"
#include "wkv7_internal.h"

namespace wkv7 {
namespace {

constexpr int kRows = 4;         // rows per lane group
constexpr int kMaxWarps = 8;
constexpr int kFirstWaveCtas = 152 * 8;  // CTAs that may start while the previous kernel drains

// How a warp covers rows of DK state entries: 16 bytes per lane.
template <int DK, bool SB>
struct Geo {
    static constexpr int kCols = SB ? 8 : 4;           // key columns per lane
    static constexpr int kLanes = DK / kCols;          // lanes per row
    static constexpr int kPer = 32 / kLanes;           // rows per warp access
    static constexpr int kWarpRows = kPer * kRows;     // rows per warp
};

template <int DK, bool SB>
int warps_for(int dv) {
    const int w = dv / Geo<DK, SB>::kWarpRows;
    return w < kMaxWarps ? w : kMaxWarps;
}

// Sums of N values over LANES consecutive lanes, value j ending in the lanes
// whose offset in the group is owner_lane<N, LANES>(j) (plus any low bits).
template <int N, int LANES>
__device__ __forceinline__ float reduce_scatter(float (&v)[N], int lane) {
    int off = LANES / 2;
#pragma unroll
    for (int n = N; n > 1; n /= 2, off /= 2) {
        const bool hi = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = hi ? v[i + n / 2] : v[i];
            const float send = hi ? v[i] : v[i + n / 2];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
#pragma unroll
    for (; off >= 1; off /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    return v[0];
}
template <int N, int LANES>
__host__ __device__ constexpr int owner_lane(int j) {
    int lane = 0, off = LANES / 2;
    for (int n = N; n > 1; n /= 2, off /= 2)
        if (j & (n / 2)) lane |= off;
    return lane;
}

// kCols state entries of one row, as floats and back.
template <bool SB, int C>
__device__ __forceinline__ void load_row(const float *base, size_t off, float (&x)[C]) {
    if constexpr (SB) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(base) + off));
        x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
        x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
    } else {
        const float4 u = __ldcs(reinterpret_cast<const float4 *>(base + off));
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    }
}
template <bool SB, int C>
__device__ __forceinline__ void store_row(float *base, size_t off, const float (&x)[C]) {
    if constexpr (SB)
        __stcs(reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(base) + off),
               make_uint4(pack_bf16_rn(x[0], x[1]), pack_bf16_rn(x[2], x[3]), pack_bf16_rn(x[4], x[5]),
                          pack_bf16_rn(x[6], x[7])));
    else
        __stcs(reinterpret_cast<float4 *>(base + off), make_float4(x[0], x[1], x[2], x[3]));
}

// kCols input values (global or shared memory) as floats.
template <bool IB, int C>
__device__ __forceinline__ void load_in(const void *p, size_t off, float (&x)[C]) {
    if constexpr (IB && C == 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + off);
        x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
        x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
    } else if constexpr (IB) {
        const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + off);
        x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
    } else {
#pragma unroll
        for (int c = 0; c < C; c += 4) {
            const float4 u = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + off + c);
            x[c] = u.x; x[c + 1] = u.y; x[c + 2] = u.z; x[c + 3] = u.w;
        }
    }
}

// What a token's heads contribute besides the rows' own sums.
struct Scalars {
    float alpha;  // exp(g)
    float beta;
    float nk;     // 1 / length of k (1 when not normalising)
    float nq;     // scale / length of q
    float kq;     // nk <k, q>
};

__device__ __forceinline__ Scalars scalars_of(float g, float beta, float kk, float qq, float kq, float scale, float eps) {
    Scalars t;
    t.alpha = expf(g);
    t.beta = beta;
    t.nk = eps > 0.f ? rsqrtf(kk + eps) : 1.f;
    t.nq = eps > 0.f ? scale * rsqrtf(qq + eps) : scale;
    t.kq = t.nk * kq;
    return t;
}

// The same with the products and sums rounded as the formulas are written (k and
// q divided by their lengths, the decayed state rounded before it is used, no
// fused multiply-add into the state): a bf16-state pool's single step.  Its new
// state is rounded to bf16, where a last-bit difference in float32 can decide
// between two neighbours 2^-8 apart, so the step keeps to the plainest order.
template <int DK, bool SB>
__device__ __forceinline__ float token_step_plain(float (&s)[kRows][Geo<DK, SB>::kCols], float (&k)[Geo<DK, SB>::kCols],
                                                  float (&q)[Geo<DK, SB>::kCols], const float (&v)[kRows], float g,
                                                  float beta, float kk, float qq, float scale, float eps, int lane) {
    using G = Geo<DK, SB>;
    const float alpha = expf(g);
    if (eps > 0.f) {
        const float lk = __fsqrt_rn(kk + eps), lq = __fsqrt_rn(qq + eps);
#pragma unroll
        for (int c = 0; c < G::kCols; ++c) {
            k[c] = __fdiv_rn(k[c], lk);
            q[c] = __fdiv_rn(q[c], lq);
        }
    }
    float sum[kRows], out[kRows];
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
        sum[m] = 0.f;
#pragma unroll
        for (int c = 0; c < G::kCols; ++c) {
            s[m][c] = __fmul_rn(s[m][c], alpha);
            sum[m] = __fadd_rn(sum[m], __fmul_rn(s[m][c], k[c]));
        }
    }
    const float mine = reduce_scatter<kRows, G::kLanes>(sum, lane);
    const int group = lane & ~(G::kLanes - 1);
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
        const float sk = __shfl_sync(0xffffffffu, mine, group | owner_lane<kRows, G::kLanes>(m));
        const float e = __fmul_rn(beta, __fsub_rn(v[m], sk));
        out[m] = 0.f;
#pragma unroll
        for (int c = 0; c < G::kCols; ++c) {
            s[m][c] = __fadd_rn(s[m][c], __fmul_rn(e, k[c]));
            out[m] = fmaf(s[m][c], q[c], out[m]);
        }
    }
    // rows scattered as token_step leaves them: the lanes' second-highest bits name the row
#pragma unroll
    for (int m = 0; m < kRows; ++m) out[m] += __shfl_xor_sync(0xffffffffu, out[m], G::kLanes / 2);
    return scale * reduce_scatter<kRows, G::kLanes / 2>(out, lane);
}

// One token on the rows a lane holds; returns, in the lanes that own it (see
// owns_out), the readout of row out_row(lane).
template <int DK, bool SB>
__device__ __forceinline__ float token_step(float (&s)[kRows][Geo<DK, SB>::kCols], const float (&k)[Geo<DK, SB>::kCols],
                                            const float (&q)[Geo<DK, SB>::kCols], const float (&v)[kRows],
                                            const Scalars &t, int lane) {
    using G = Geo<DK, SB>;
    float sum[2 * kRows];
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int c = 0; c < G::kCols; ++c) {
            a = fmaf(s[m][c], k[c], a);
            b = fmaf(s[m][c], q[c], b);
        }
        sum[m] = a;
        sum[kRows + m] = b;
    }
    const float mine = reduce_scatter<2 * kRows, G::kLanes>(sum, lane);
    const int group = lane & ~(G::kLanes - 1);
    float e[kRows];
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
        const float sk = __shfl_sync(0xffffffffu, mine, group | owner_lane<2 * kRows, G::kLanes>(m));
        e[m] = t.beta * (v[m] - t.alpha * t.nk * sk);
        const float ek = e[m] * t.nk;
#pragma unroll
        for (int c = 0; c < G::kCols; ++c) s[m][c] = fmaf(t.alpha, s[m][c], ek * k[c]);
    }
    const bool b1 = (lane & (G::kLanes / 4)) != 0, b0 = (lane & (G::kLanes / 8)) != 0;
    const float em = b1 ? (b0 ? e[3] : e[2]) : (b0 ? e[1] : e[0]);
    return t.nq * fmaf(t.alpha, mine, em * t.kq);
}
// A lane that ends with a readout, and the row (of its warp's) it is for.
template <int DK, bool SB>
__device__ __forceinline__ bool owns_out(int lane) {
    constexpr int L = Geo<DK, SB>::kLanes;
    return (lane & (L / 2)) != 0 && (lane & (L / 8 - 1)) == 0;
}
template <int DK, bool SB>
__device__ __forceinline__ int out_row(int lane) {
    using G = Geo<DK, SB>;
    const int m = ((lane & (G::kLanes / 4)) ? 2 : 0) + ((lane & (G::kLanes / 8)) ? 1 : 0);
    return m * G::kPer + lane / G::kLanes;
}

// ------------------------------------------------------------------- decode

// One CTA advances up to 8 warps' rows of one (batch row, value head).  Like the
// WKV-7 decode it reads its slot id and warms L2 with its rows before it waits
// for the previous kernel.
template <int DK, bool SB, bool IB>
__global__ void __launch_bounds__(32 * kMaxWarps) gdn_decode_kernel(const GdnDecodeArgs p, int tiles) {
    using G = Geo<DK, SB>;
    pdl_launch_dependents();
    const int unit = blockIdx.x / tiles, tile = blockIdx.x - unit * tiles;
    const int bi = unit / p.lv.hv, h = unit - bi * p.lv.hv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = tile * (blockDim.x >> 5) * G::kWarpRows + warp * G::kWarpRows;  // this warp's first row
    const int r = row0 + lane / G::kLanes;                                           // this lane's first row
    const int c = (lane & (G::kLanes - 1)) * G::kCols;
    const int slot = __ldg(p.slot_ids + bi);
    const bool ok = slot >= 0 && slot < p.lv.n_slots;
    const size_t s_off = static_cast<size_t>(ok ? slot : 0) * p.lv.slot_stride + p.lv.layer_off +
                         static_cast<size_t>(h) * p.lv.dv * DK + c;
    if (ok && blockIdx.x < kFirstWaveCtas && (lane & 7) == 0) {  // one prefetch per 128-byte line
#pragma unroll
        for (int m = 0; m < kRows; ++m) {
            const size_t off = s_off + static_cast<size_t>(r + m * G::kPer) * DK;
            prefetch_l2(SB ? static_cast<const void *>(reinterpret_cast<const uint16_t *>(p.lv.states) + off)
                           : static_cast<const void *>(p.lv.states + off));
        }
    }
    pdl_wait();
    if (!ok) {
        if (threadIdx.x == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SLOT);
        return;
    }
    float s[kRows][G::kCols];
#pragma unroll
    for (int m = 0; m < kRows; ++m) load_row<SB>(p.lv.states, s_off + static_cast<size_t>(r + m * G::kPer) * DK, s[m]);
    const int hk = h / (p.lv.hv / p.lv.hk);
    float k[G::kCols], q[G::kCols], v[kRows];
    load_in<IB>(p.in.k, static_cast<size_t>(bi) * p.in.k_stride + static_cast<size_t>(hk) * DK + c, k);
    load_in<IB>(p.in.q, static_cast<size_t>(bi) * p.in.q_stride + static_cast<size_t>(hk) * DK + c, q);
#pragma unroll
    for (int m = 0; m < kRows; ++m)
        v[m] = load1<IB>(p.in.v, static_cast<size_t>(bi) * p.in.v_stride + static_cast<size_t>(h) * p.lv.dv + r +
                                     m * G::kPer);
    const float g = __ldg(p.in.g + static_cast<size_t>(bi) * p.in.g_stride + h);
    const float beta = __ldg(p.in.beta + static_cast<size_t>(bi) * p.in.beta_stride + h);
    float dots[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < G::kCols; ++x) {
        dots[0] = fmaf(k[x], k[x], dots[0]);
        dots[1] = fmaf(q[x], q[x], dots[1]);
        dots[2] = fmaf(k[x], q[x], dots[2]);
    }
    const float d = reduce_scatter<4, G::kLanes>(dots, lane);
    const int group = lane & ~(G::kLanes - 1);
    const float kk = __shfl_sync(0xffffffffu, d, group | owner_lane<4, G::kLanes>(0));
    const float qq = __shfl_sync(0xffffffffu, d, group | owner_lane<4, G::kLanes>(1));
    const float kq = __shfl_sync(0xffffffffu, d, group | owner_lane<4, G::kLanes>(2));
    float o;
    if constexpr (SB)
        o = token_step_plain<DK, SB>(s, k, q, v, g, beta, kk, qq, p.in.scale, p.in.eps, lane);
    else
        o = token_step<DK, SB>(s, k, q, v, scalars_of(g, beta, kk, qq, kq, p.in.scale, p.in.eps), lane);
#pragma unroll
    for (int m = 0; m < kRows; ++m) store_row<SB>(p.lv.states, s_off + static_cast<size_t>(r + m * G::kPer) * DK, s[m]);
    if (owns_out<DK, SB>(lane))
        store_out(p.in.o, p.in.o_bf16, static_cast<size_t>(unit) * p.lv.dv + row0 + out_row<DK, SB>(lane), o);
}

// ------------------------------------------------------------ runs of tokens

constexpr int kGroup = 16;  // tokens staged per pass

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async4(void *dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// Staged inputs of one group of tokens, as they come.
template <int DK, bool IB>
struct Stage {
    using Elem = typename std::conditional<IB, uint16_t, float>::type;
    Elem k[kGroup][DK], q[kGroup][DK];
    Elem v[kGroup][kMaxWarps * Geo<DK, true>::kWarpRows];  // the tile's rows (bf16 states have the larger tiles)
    float g[kGroup], beta[kGroup];
};

// A run of tokens on the rows of one CTA, held in registers throughout.  The
// inputs of 16 tokens are staged at a time, the next 16 arriving meanwhile; the
// dot products that every row shares (lengths, <k, q>) are taken once per token
// by one warp.  With step_snap_ids the state after every token is streamed to its
// snapshot.  A bf16-state pool rounds after every token of a multi-token decode
// (K single steps), and only where a state is stored in a prefill.
template <int DK, bool SB, bool IB>
__global__ void __launch_bounds__(32 * kMaxWarps) gdn_run_kernel(const GdnRunArgs p, int tiles) {
    using G = Geo<DK, SB>;
    __shared__ __align__(16) Stage<DK, IB> st[2];
    __shared__ Scalars sc[kGroup];
    pdl_prologue();
    const int unit = blockIdx.x / tiles, tile = blockIdx.x - unit * tiles;
    const int bi = unit / p.lv.hv, h = unit - bi * p.lv.hv;
    const int warps = blockDim.x >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile_rows = warps * G::kWarpRows;
    const int r = warp * G::kWarpRows + lane / G::kLanes;  // this lane's first row in the tile
    const int c = (lane & (G::kLanes - 1)) * G::kCols;
    const int slot = __ldg(p.slot_ids + bi);
    if (slot < 0 || slot >= p.lv.n_slots) {
        if (threadIdx.x == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SLOT);
        return;
    }
    long long t0 = static_cast<long long>(bi) * p.n_tok;
    int len = p.n_tok, ck0 = 0;
    if (p.cu_seqlens) {
        const int a = __ldg(p.cu_seqlens + bi), b = __ldg(p.cu_seqlens + bi + 1);
        bool bad = a < 0 || b < a || b > p.total_tokens || b - a > p.max_seqlen;
        if (!bad && p.cu_ckpt) {
            ck0 = __ldg(p.cu_ckpt + bi);
            bad = ck0 < 0 || __ldg(p.cu_ckpt + bi + 1) - ck0 != (b - a) / 64;
        }
        if (bad) {
            if (threadIdx.x == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SEQLENS);
            return;
        }
        t0 = a;
        len = b - a;
        if (len == 0) return;
    }
    const size_t head_off = p.lv.layer_off + (static_cast<size_t>(h) * p.lv.dv + static_cast<size_t>(tile) * tile_rows) * DK + c;
    const size_t s_off = static_cast<size_t>(slot) * p.lv.slot_stride + head_off;
    float s[kRows][G::kCols];
#pragma unroll
    for (int m = 0; m < kRows; ++m) load_row<SB>(p.lv.states, s_off + static_cast<size_t>(r + m * G::kPer) * DK, s[m]);

    const int hk = h / (p.lv.hv / p.lv.hk);
    using Elem = typename Stage<DK, IB>::Elem;
    auto stage = [&](int buf, int first) {
        Stage<DK, IB> &d = st[buf];
        const int n = min(kGroup, len - first);
        constexpr int kChunk = 16 / static_cast<int>(sizeof(Elem));  // elements per 16 bytes
        constexpr int kKey = DK / kChunk;
        const int vc = tile_rows / kChunk, per = 2 * kKey + vc;
        for (int e = threadIdx.x; e < n * per; e += blockDim.x) {
            const int t = e / per, x = e - t * per;
            const long long row = t0 + first + t;
            if (x < kKey)
                cp_async16(&d.k[t][x * kChunk], static_cast<const Elem *>(p.in.k) + row * p.in.k_stride +
                                                    static_cast<long long>(hk) * DK + x * kChunk);
            else if (x < 2 * kKey)
                cp_async16(&d.q[t][(x - kKey) * kChunk], static_cast<const Elem *>(p.in.q) + row * p.in.q_stride +
                                                             static_cast<long long>(hk) * DK + (x - kKey) * kChunk);
            else
                cp_async16(&d.v[t][(x - 2 * kKey) * kChunk],
                           static_cast<const Elem *>(p.in.v) + row * p.in.v_stride +
                               static_cast<long long>(h) * p.lv.dv + tile * tile_rows + (x - 2 * kKey) * kChunk);
        }
        if (threadIdx.x < 2 * n) {
            const int t = threadIdx.x >> 1;
            const long long row = t0 + first + t;
            if (threadIdx.x & 1)
                cp_async4(&d.beta[t], p.in.beta + row * p.in.beta_stride + h);
            else
                cp_async4(&d.g[t], p.in.g + row * p.in.g_stride + h);
        }
    };
    stage(0, 0);
    cp_async_commit();
    const bool round_each = SB && p.cu_seqlens == nullptr;
#pragma unroll 1
    for (int first = 0, buf = 0; first < len; first += kGroup, buf ^= 1) {
        const int n = min(kGroup, len - first);
        if (first + kGroup < len) stage(buf ^ 1, first + kGroup);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        const Stage<DK, IB> &d = st[buf];
        for (int t = warp; t < n; t += warps) {  // the sums that every row shares
            float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
            for (int x = 0; x < DK; x += 32) {
                const float a = widen(d.k[t][x + lane]), b = widen(d.q[t][x + lane]);
                kk = fmaf(a, a, kk);
                qq = fmaf(b, b, qq);
                kq = fmaf(a, b, kq);
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) {
                kk += __shfl_xor_sync(0xffffffffu, kk, off);
                qq += __shfl_xor_sync(0xffffffffu, qq, off);
                kq += __shfl_xor_sync(0xffffffffu, kq, off);
            }
            if (lane == 0) sc[t] = scalars_of(d.g[t], d.beta[t], kk, qq, kq, p.in.scale, p.in.eps);
        }
        __syncthreads();
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
            float k[G::kCols], q[G::kCols], v[kRows];
            load_in<IB>(d.k[t], c, k);
            load_in<IB>(d.q[t], c, q);
#pragma unroll
            for (int m = 0; m < kRows; ++m) v[m] = widen(d.v[t][r + m * G::kPer]);
            const float o = token_step<DK, SB>(s, k, q, v, sc[t], lane);
            const long long row = t0 + first + t;
            if (owns_out<DK, SB>(lane))
                store_out(p.in.o, p.in.o_bf16,
                          (static_cast<size_t>(row) * p.lv.hv + h) * p.lv.dv + tile * tile_rows +
                              warp * G::kWarpRows + out_row<DK, SB>(lane),
                          o);
            const int done = first + t + 1;
            int id = 0;
            const bool boundary = p.cu_ckpt && done % 64 == 0;
            if (round_each || boundary) {
                if constexpr (SB) {
#pragma unroll
                    for (int m = 0; m < kRows; ++m)
#pragma unroll
                        for (int x = 0; x < G::kCols; ++x) s[m][x] = round_bf16(s[m][x]);
                }
            }
            if (p.step_snap_ids)
                id = __ldg(p.step_snap_ids + row);
            else if (boundary)
                id = __ldg(p.ckpt_ids + ck0 + done / 64 - 1);
            else
                continue;
            if (id < 0 || id >= p.lv.n_snaps) {
                if (threadIdx.x == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SLOT);
                continue;
            }
            const size_t d_off = static_cast<size_t>(id) * p.lv.slot_stride + head_off;
#pragma unroll
            for (int m = 0; m < kRows; ++m)
                store_row<SB>(p.lv.snaps, d_off + static_cast<size_t>(r + m * G::kPer) * DK, s[m]);
        }
        __syncthreads();  // this buffer is refilled by the next pass
    }
#pragma unroll
    for (int m = 0; m < kRows; ++m) store_row<SB>(p.lv.states, s_off + static_cast<size_t>(r + m * G::kPer) * DK, s[m]);
}

template <int DK, bool SB, bool IB>
cudaError_t decode_as(const GdnDecodeArgs &a, cudaStream_t s) {
    const int warps = warps_for<DK, SB>(a.lv.dv), tiles = a.lv.dv / (warps * Geo<DK, SB>::kWarpRows);
    const long long ctas = static_cast<long long>(a.n) * a.lv.hv * tiles;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(gdn_decode_kernel<DK, SB, IB>, dim3(static_cast<unsigned>(ctas)), dim3(32 * warps), 0, s, a, tiles);
}

template <int DK, bool SB, bool IB>
cudaError_t run_as(const GdnRunArgs &a, cudaStream_t s) {
    const int warps = warps_for<DK, SB>(a.lv.dv), tiles = a.lv.dv / (warps * Geo<DK, SB>::kWarpRows);
    const long long ctas = static_cast<long long>(a.n) * a.lv.hv * tiles;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(gdn_run_kernel<DK, SB, IB>, dim3(static_cast<unsigned>(ctas)), dim3(32 * warps), 0, s, a, tiles);
}

}  // namespace

cudaError_t launch_gdn_decode(const GdnDecodeArgs &a, cudaStream_t s, int *launches) {
    cudaError_t (*const as[8])(const GdnDecodeArgs &, cudaStream_t) = {
        decode_as<64, false, false>,  decode_as<64, false, true>,  decode_as<64, true, false>,  decode_as<64, true, true>,
        decode_as<128, false, false>, decode_as<128, false, true>, decode_as<128, true, false>, decode_as<128, true, true>};
    const cudaError_t e = as[(a.lv.dk == 128 ? 4 : 0) | (a.lv.state_bf16 ? 2 : 0) | (a.in.bf16 ? 1 : 0)](a, s);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_gdn_run(const GdnRunArgs &a, cudaStream_t s, int *launches) {
    cudaError_t (*const as[8])(const GdnRunArgs &, cudaStream_t) = {
        run_as<64, false, false>,  run_as<64, false, true>,  run_as<64, true, false>,  run_as<64, true, true>,
        run_as<128, false, false>, run_as<128, false, true>, run_as<128, true, false>, run_as<128, true, true>};
    const cudaError_t e = as[(a.lv.dk == 128 ? 4 : 0) | (a.lv.state_bf16 ? 2 : 0) | (a.in.bf16 ? 1 : 0)](a, s);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace wkv7
