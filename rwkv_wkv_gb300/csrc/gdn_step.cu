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
// the launch and three dependent reads.  With bf16 states the step's rounding rule costs
// instructions (token_step_plain): 201 slots of 12 heads of 64, 40 MB that stay in L2, 7.9 us (8.3
// before its products went in pairs), 256 of 32 heads of 128, 0.55 GB, 107 us (5.1 TB/s).  A run with a state to keep after each token is bound by writing them: 48 slots x
// 5 tokens x 32 heads, 0.71 GB, 106 us (6.7 TB/s; bf16 states 70); without them by the shuffles and
// the inputs' staging (66 us, bf16 states 60; 1 sequence of 24 tokens 14.7 us, of 128 86, on
// bf16 states 64).
#include <type_traits>

#include "device_common.cuh"
#include "packed_f32.cuh"
#include "wkv7_internal.h"

namespace wkv7 {
namespace {

constexpr int kRows = 4;         // rows per lane group
constexpr int kMaxWarps = 8;
constexpr int kFirstWaveCtas = 152 * 8;  // CTAs that may start while the previous kernel drains

// How a warp covers rows of DK state entries: 16 bytes per lane, consecutive columns (kRun = kCols).
// Where a bf16-state pool steps token by token (ST, "strided") a lane holds kRun columns of every
// 32 instead: columns c, c + 32, ... meet in one lane, where that step's sums begin (token_step_plain).
// Runs of a prefill keep to 16 bytes: 1 sequence of 128 tokens, heads of 128, 63 us, 89 strided.
template <int DK, bool SB, bool ST = false>
struct Geo {
    static constexpr int kCols = SB ? 8 : 4;           // key columns per lane
    static constexpr int kLanes = DK / kCols;          // lanes per row
    static constexpr int kPer = 32 / kLanes;           // rows per warp access
    static constexpr int kWarpRows = kPer * kRows;     // rows per warp
    static constexpr int kRun = ST ? 32 / kLanes : kCols;  // consecutive columns of a lane ...
    static constexpr int kPieces = kCols / kRun;           // ... in each of so many ranges of 32
    static __device__ __forceinline__ int column(int lane) { return (lane & (kLanes - 1)) * kRun; }  // a lane's first
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

// C consecutive bf16 values at p, as floats and back.
template <int C>
__device__ __forceinline__ void unpack_bf16(const uint32_t (&u)[C / 2], float *x) {
#pragma unroll
    for (int i = 0; i < C / 2; ++i) x[2 * i] = bf16_lo(u[i]), x[2 * i + 1] = bf16_hi(u[i]);
}
template <int C>
__device__ __forceinline__ void load_bf16(const uint16_t *p, float *x) {
    if constexpr (C == 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        unpack_bf16<8>({u.x, u.y, u.z, u.w}, x);
    } else if constexpr (C == 4) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        unpack_bf16<4>({u.x, u.y}, x);
    } else {
        unpack_bf16<2>({*reinterpret_cast<const uint32_t *>(p)}, x);
    }
}

// A lane's state entries of one row, the first at `off`, as floats and back.
template <class G, bool SB>
__device__ __forceinline__ void load_row(const float *base, size_t off, float (&x)[G::kCols]) {
    if constexpr (SB) {
        const uint16_t *at = reinterpret_cast<const uint16_t *>(base) + off;
#pragma unroll
        for (int m = 0; m < G::kPieces; ++m) {
            float *y = x + m * G::kRun;
            if constexpr (G::kRun == 8) {
                const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(at));
                unpack_bf16<8>({u.x, u.y, u.z, u.w}, y);
            } else if constexpr (G::kRun == 4) {
                const uint2 u = __ldcs(reinterpret_cast<const uint2 *>(at + 32 * m));
                unpack_bf16<4>({u.x, u.y}, y);
            } else {
                unpack_bf16<2>({__ldcs(reinterpret_cast<const uint32_t *>(at + 32 * m))}, y);
            }
        }
    } else {
        const float4 u = __ldcs(reinterpret_cast<const float4 *>(base + off));
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    }
}
template <class G, bool SB>
__device__ __forceinline__ void store_row(float *base, size_t off, const float (&x)[G::kCols]) {
    if constexpr (SB) {
        uint16_t *at = reinterpret_cast<uint16_t *>(base) + off;
#pragma unroll
        for (int m = 0; m < G::kPieces; ++m) {
            const float *y = x + m * G::kRun;
            if constexpr (G::kRun == 8)
                __stcs(reinterpret_cast<uint4 *>(at), make_uint4(pack_bf16_rn(y[0], y[1]), pack_bf16_rn(y[2], y[3]),
                                                                 pack_bf16_rn(y[4], y[5]), pack_bf16_rn(y[6], y[7])));
            else if constexpr (G::kRun == 4)
                __stcs(reinterpret_cast<uint2 *>(at + 32 * m), make_uint2(pack_bf16_rn(y[0], y[1]), pack_bf16_rn(y[2], y[3])));
            else
                __stcs(reinterpret_cast<uint32_t *>(at + 32 * m), pack_bf16_rn(y[0], y[1]));
        }
    } else {
        __stcs(reinterpret_cast<float4 *>(base + off), make_float4(x[0], x[1], x[2], x[3]));
    }
}

// The same columns of an input row (global or shared memory) as floats.
template <class G, bool IB>
__device__ __forceinline__ void load_in(const void *p, size_t off, float (&x)[G::kCols]) {
#pragma unroll
    for (int m = 0; m < G::kPieces; ++m) {
        float *y = x + m * G::kRun;
        const size_t at = off + 32 * m;
        if constexpr (IB) {
            load_bf16<G::kRun>(static_cast<const uint16_t *>(p) + at, y);
        } else if constexpr (G::kRun >= 4) {
#pragma unroll
            for (int c = 0; c < G::kRun; c += 4) {
                const float4 u = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at + c);
                y[c] = u.x; y[c + 1] = u.y; y[c + 2] = u.z; y[c + 3] = u.w;
            }
        } else {
            const float2 u = *reinterpret_cast<const float2 *>(static_cast<const float *>(p) + at);
            y[0] = u.x; y[1] = u.y;
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

__device__ __forceinline__ float q_factor(float qq, float scale, float eps) {
    return eps > 0.f ? __fmul_rn(scale, rsqrtf(__fadd_rn(qq, eps))) : scale;
}
__device__ __forceinline__ Scalars scalars_of(float g, float beta, float kk, float qq, float kq, float scale, float eps) {
    Scalars t;
    t.alpha = expf(g);
    t.beta = beta;
    t.nk = eps > 0.f ? rsqrtf(__fadd_rn(kk, eps)) : 1.f;
    t.nq = q_factor(qq, scale, eps);
    t.kq = __fmul_rn(t.nk, kq);
    return t;
}

// A sum rounded on its own.  (The packed addition of a packed product comes out fused for some
// operands, the length of float32 keys among them, whatever its rounding modifier; the scalar one
// keeps to it.  Products stay packed.)
__device__ __forceinline__ F2 add_rn(F2 a, F2 b) {
    float x, y, z, w;
    unpack(a, x, y);
    unpack(b, z, w);
    return f2(__fadd_rn(x, z), __fadd_rn(y, w));
}
// A lane's part of a bf16-state row's sum: its products, rounded, those 32 columns apart first, then neighbours.
template <int DK>
__device__ __forceinline__ float lane_sum(const F2 (&a)[4], const F2 (&b)[4]) {
    static_assert(Geo<DK, true, true>::kCols == 8, "");
    F2 p = a[0] * b[0];
    float x, y;
    if constexpr (Geo<DK, true, true>::kRun == 4) {
        p = add_rn(p, a[2] * b[2]);
        F2 r = a[1] * b[1];
        r = add_rn(r, a[3] * b[3]);
        float z, w;
        unpack(p, x, y);
        unpack(r, z, w);
        return __fadd_rn(__fadd_rn(x, y), __fadd_rn(z, w));
    } else {
#pragma unroll
        for (int m = 1; m < 4; ++m) p = add_rn(p, a[m] * b[m]);
        unpack(p, x, y);
        return __fadd_rn(x, y);
    }
}
template <int C>
__device__ __forceinline__ void pack_pairs(const float (&x)[C], F2 (&y)[C / 2]) {
#pragma unroll
    for (int i = 0; i < C / 2; ++i) y[i] = f2(x[2 * i], x[2 * i + 1]);
}
// A sum over a row's lanes, neighbours first; every lane gets it.
template <int LANES>
__device__ __forceinline__ float sum_lanes(float x) {
#pragma unroll
    for (int off = 1; off < LANES; off *= 2) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, off));
    return x;
}

// The step of a bf16-state pool's decode: products, sums, quotients and the root rounded one by
// one as the formulas are written (k divided by its length, the decayed state rounded before it
// is used, no fused multiply-add into the state), and the sums over columns in one fixed order:
// x_c + x_{c+32} (+ x_{c+64} + x_{c+96}) for c < 32, then a binary tree of neighbours.  The new
// state is rounded to bf16, where a last-bit difference of two float32 results can decide between
// neighbours 2^-8 apart, so "agrees to float32 rounding" would not hold from the second step on; what
// holds is that anyone who evaluates the formulas in this order (elementary float32 operations
// and a strided 32-lane sum do) has the stored bits.  Only o, which is not carried on, is taken
// in another order and with q's length as a factor.
template <int DK>
__device__ __forceinline__ float token_step_plain(float (&s)[kRows][Geo<DK, true, true>::kCols],
                                                  const float (&k)[Geo<DK, true, true>::kCols],
                                                  const float (&q)[Geo<DK, true, true>::kCols], const float (&v)[kRows], float alpha,
                                                  float beta, float nq, int lane) {
    using G = Geo<DK, true, true>;
    constexpr int P = G::kCols / 2;
    float sum[kRows], out[kRows];
    F2 x[kRows][P], k2[P], q2[P];
    pack_pairs(k, k2);
    pack_pairs(q, q2);
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
        pack_pairs(s[m], x[m]);
#pragma unroll
        for (int c = 0; c < P; ++c) x[m][c] = x[m][c] * f2(alpha, alpha);
        sum[m] = lane_sum<DK>(x[m], k2);
    }
    // four rows' sums scattered over the lanes' two low bits, then summed over the other bits
    const bool b0 = (lane & 1) != 0, b1 = (lane & 2) != 0;
    const float x0 = __fadd_rn(b0 ? sum[2] : sum[0], __shfl_xor_sync(0xffffffffu, b0 ? sum[0] : sum[2], 1));
    const float x1 = __fadd_rn(b0 ? sum[3] : sum[1], __shfl_xor_sync(0xffffffffu, b0 ? sum[1] : sum[3], 1));
    float mine = __fadd_rn(b1 ? x1 : x0, __shfl_xor_sync(0xffffffffu, b1 ? x0 : x1, 2));
#pragma unroll
    for (int off = 4; off < G::kLanes; off *= 2) mine = __fadd_rn(mine, __shfl_xor_sync(0xffffffffu, mine, off));
    const int group = lane & ~(G::kLanes - 1);
#pragma unroll
    for (int m = 0; m < kRows; ++m) {
        const float sk = __shfl_sync(0xffffffffu, mine, group | (m >> 1) | ((m & 1) << 1));
        const float e = __fmul_rn(beta, __fsub_rn(v[m], sk));
        F2 o2 = f2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < P; ++c) {
            x[m][c] = add_rn(x[m][c], f2(e, e) * k2[c]);
            unpack(x[m][c], s[m][2 * c], s[m][2 * c + 1]);
            o2 = fma2(x[m][c], q2[c], o2);
        }
        float lo, hi;
        unpack(o2, lo, hi);
        out[m] = lo + hi;
    }
    // rows scattered as token_step leaves them: the lanes' second-highest bits name the row
#pragma unroll
    for (int m = 0; m < kRows; ++m) out[m] += __shfl_xor_sync(0xffffffffu, out[m], G::kLanes / 2);
    return __fmul_rn(nq, reduce_scatter<kRows, G::kLanes / 2>(out, lane));
}

// A token's scalars from the lanes' columns of k and q.  Decode and runs of tokens both come here, and
// neither this nor token_step leaves the compiler a choice of roundings: K tokens of a run
// leave the bits of K single steps.
template <int DK, bool SB>
__device__ __forceinline__ Scalars head_scalars(const float (&k)[Geo<DK, SB>::kCols], const float (&q)[Geo<DK, SB>::kCols],
                                                float g, float beta, float scale, float eps, int lane) {
    using G = Geo<DK, SB>;
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
    return scalars_of(g, beta, kk, qq, kq, scale, eps);
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
        e[m] = __fmul_rn(t.beta, fmaf(-__fmul_rn(t.alpha, t.nk), sk, v[m]));
        const float ek = __fmul_rn(e[m], t.nk);
#pragma unroll
        for (int c = 0; c < G::kCols; ++c) s[m][c] = fmaf(t.alpha, s[m][c], __fmul_rn(ek, k[c]));
    }
    const bool b1 = (lane & (G::kLanes / 4)) != 0, b0 = (lane & (G::kLanes / 8)) != 0;
    const float em = b1 ? (b0 ? e[3] : e[2]) : (b0 ? e[1] : e[0]);
    return __fmul_rn(t.nq, fmaf(t.alpha, mine, __fmul_rn(em, t.kq)));
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
    using G = Geo<DK, SB, SB>;
    pdl_launch_dependents();
    const int unit = blockIdx.x / tiles, tile = blockIdx.x - unit * tiles;
    const int bi = unit / p.lv.hv, h = unit - bi * p.lv.hv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = tile * (blockDim.x >> 5) * G::kWarpRows + warp * G::kWarpRows;  // this warp's first row
    const int r = row0 + lane / G::kLanes;                                           // this lane's first row
    const int c = G::column(lane);
    const int slot = __ldg(p.slot_ids + bi);
    const bool ok = slot >= 0 && slot < p.lv.n_slots;
    const size_t s_off = static_cast<size_t>(ok ? slot : 0) * p.lv.slot_stride + p.lv.layer_off +
                         static_cast<size_t>(h) * p.lv.dv * DK + c;
    if (ok && blockIdx.x < kFirstWaveCtas && (lane & 7) == 0) {  // one prefetch per 128-byte line
        const int line = SB ? (lane & (G::kLanes - 1)) * (G::kCols - G::kRun) : 0;  // from the lane's column to its line
#pragma unroll
        for (int m = 0; m < kRows; ++m) {
            const size_t off = s_off + static_cast<size_t>(r + m * G::kPer) * DK + line;
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
    for (int m = 0; m < kRows; ++m) load_row<G, SB>(p.lv.states, s_off + static_cast<size_t>(r + m * G::kPer) * DK, s[m]);
    const int hk = h / (p.lv.hv / p.lv.hk);
    float k[G::kCols], q[G::kCols], v[kRows];
    load_in<G, IB>(p.in.k, static_cast<size_t>(bi) * p.in.k_stride + static_cast<size_t>(hk) * DK + c, k);
    load_in<G, IB>(p.in.q, static_cast<size_t>(bi) * p.in.q_stride + static_cast<size_t>(hk) * DK + c, q);
#pragma unroll
    for (int m = 0; m < kRows; ++m)
        v[m] = load1<IB>(p.in.v, static_cast<size_t>(bi) * p.in.v_stride + static_cast<size_t>(h) * p.lv.dv + r +
                                     m * G::kPer);
    const float g = __ldg(p.in.g + static_cast<size_t>(bi) * p.in.g_stride + h);
    const float beta = __ldg(p.in.beta + static_cast<size_t>(bi) * p.in.beta_stride + h);
    float o;
    if constexpr (SB) {
        F2 k2[G::kCols / 2], q2[G::kCols / 2];
        pack_pairs(k, k2);
        pack_pairs(q, q2);
        const float kk = sum_lanes<G::kLanes>(lane_sum<DK>(k2, k2)), qq = sum_lanes<G::kLanes>(lane_sum<DK>(q2, q2));
        const float lk = __fsqrt_rn(__fadd_rn(kk, p.in.eps));
        if (p.in.eps > 0.f) {
#pragma unroll
            for (int x = 0; x < G::kCols; ++x) k[x] = __fdiv_rn(k[x], lk);
        }
        o = token_step_plain<DK>(s, k, q, v, expf(g), beta, q_factor(qq, p.in.scale, p.in.eps), lane);
    } else {
        o = token_step<DK, SB>(s, k, q, v, head_scalars<DK, SB>(k, q, g, beta, p.in.scale, p.in.eps, lane), lane);
    }
#pragma unroll
    for (int m = 0; m < kRows; ++m) store_row<G, SB>(p.lv.states, s_off + static_cast<size_t>(r + m * G::kPer) * DK, s[m]);
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
// snapshot.  A multi-token decode leaves the bits of K single steps; on a bf16-state pool (STEPS)
// it takes decode's step, rounded after every token, with k / |k| and q laid out in float32 beside
// the sums as token_step_plain's lanes hold them.  A prefill rounds only where a state is stored.
// (STEPS wants four CTAs an SM: 48 slots x 5 tokens of 32 heads of 128 with every state kept 70 us, over 73
// with three.  The others are best left to the compiler, 56 to 80 registers.)
template <int DK, bool SB, bool IB, bool STEPS>
__global__ void __launch_bounds__(32 * kMaxWarps, STEPS ? 4 : 0) gdn_run_kernel(const GdnRunArgs p, int tiles) {
    static_assert(SB || !STEPS, "float32 states take token_step throughout");
    using G = Geo<DK, SB, STEPS>;
    __shared__ __align__(16) Stage<DK, IB> st[2];
    __shared__ Scalars sc[kGroup];
    // STEPS: a token's k / |k| and q; float32 inputs are replaced where they were staged
    __shared__ __align__(16) float unit_kq[STEPS && IB ? 2 * kGroup : 1][STEPS && IB ? DK : 4];
    pdl_prologue();
    const int unit = blockIdx.x / tiles, tile = blockIdx.x - unit * tiles;
    const int bi = unit / p.lv.hv, h = unit - bi * p.lv.hv;
    const int warps = blockDim.x >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile_rows = warps * G::kWarpRows;
    const int r = warp * G::kWarpRows + lane / G::kLanes;  // this lane's first row in the tile
    const int c = G::column(lane);
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
    for (int m = 0; m < kRows; ++m) load_row<G, SB>(p.lv.states, s_off + static_cast<size_t>(r + m * G::kPer) * DK, s[m]);

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
    auto unit_k = [&](int buf, int t) { return IB ? unit_kq[2 * t] : reinterpret_cast<float *>(st[buf].k[t]); };
    auto unit_q = [&](int buf, int t) { return IB ? unit_kq[2 * t + 1] : reinterpret_cast<float *>(st[buf].q[t]); };
#pragma unroll 1
    for (int first = 0, buf = 0; first < len; first += kGroup, buf ^= 1) {
        const int n = min(kGroup, len - first);
        if (first + kGroup < len) stage(buf ^ 1, first + kGroup);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        const Stage<DK, IB> &d = st[buf];
        for (int t = warp; t < n; t += warps) {  // the sums that every row shares
            if constexpr (STEPS) {
                constexpr int kRanges = DK / 32;
                float kx[kRanges], qx[kRanges];
#pragma unroll
                for (int m = 0; m < kRanges; ++m) kx[m] = widen(d.k[t][32 * m + lane]), qx[m] = widen(d.q[t][32 * m + lane]);
                float kk = __fmul_rn(kx[0], kx[0]), qq = __fmul_rn(qx[0], qx[0]);
#pragma unroll
                for (int m = 1; m < kRanges; ++m)
                    kk = __fadd_rn(kk, __fmul_rn(kx[m], kx[m])), qq = __fadd_rn(qq, __fmul_rn(qx[m], qx[m]));
                kk = sum_lanes<32>(kk), qq = sum_lanes<32>(qq);
                const float lk = __fsqrt_rn(__fadd_rn(kk, p.in.eps));
                __syncwarp();
#pragma unroll
                for (int m = 0; m < kRanges; ++m) {  // entry m * kRun + lane % kRun of lane / kRun's: 4 of each lane, then the other 4
                    const int e = m * G::kRun + lane % G::kRun, at = e / 4 * (4 * G::kLanes) + lane / G::kRun * 4 + e % 4;
                    unit_k(buf, t)[at] = p.in.eps > 0.f ? __fdiv_rn(kx[m], lk) : kx[m];
                    unit_q(buf, t)[at] = qx[m];
                }
                if (lane == 0) {
                    sc[t].alpha = expf(d.g[t]);
                    sc[t].beta = d.beta[t];
                    sc[t].nq = q_factor(qq, p.in.scale, p.in.eps);
                }
            } else if constexpr (!SB) {
                float k[G::kCols], q[G::kCols];
                load_in<G, IB>(d.k[t], c, k);
                load_in<G, IB>(d.q[t], c, q);
                const Scalars x = head_scalars<DK, SB>(k, q, d.g[t], d.beta[t], p.in.scale, p.in.eps, lane);
                if (lane == 0) sc[t] = x;
            } else {
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
        }
        __syncthreads();
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
            float k[G::kCols], q[G::kCols], v[kRows];
#pragma unroll
            for (int m = 0; m < kRows; ++m) v[m] = widen(d.v[t][r + m * G::kPer]);
            float o;
            if constexpr (STEPS) {
                const int at = (lane & (G::kLanes - 1)) * 4;
#pragma unroll
                for (int x = 0; x < G::kCols; x += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(unit_k(buf, t) + x * G::kLanes + at);
                    const float4 b = *reinterpret_cast<const float4 *>(unit_q(buf, t) + x * G::kLanes + at);
                    k[x] = a.x, k[x + 1] = a.y, k[x + 2] = a.z, k[x + 3] = a.w;
                    q[x] = b.x, q[x + 1] = b.y, q[x + 2] = b.z, q[x + 3] = b.w;
                }
                o = token_step_plain<DK>(s, k, q, v, sc[t].alpha, sc[t].beta, sc[t].nq, lane);
            } else {
                load_in<G, IB>(d.k[t], c, k);
                load_in<G, IB>(d.q[t], c, q);
                o = token_step<DK, SB>(s, k, q, v, sc[t], lane);
            }
            const long long row = t0 + first + t;
            if (owns_out<DK, SB>(lane))
                store_out(p.in.o, p.in.o_bf16,
                          (static_cast<size_t>(row) * p.lv.hv + h) * p.lv.dv + tile * tile_rows +
                              warp * G::kWarpRows + out_row<DK, SB>(lane),
                          o);
            const int done = first + t + 1;
            int id = 0;
            const bool boundary = p.cu_ckpt && done % 64 == 0;
            if (STEPS || boundary) {
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
                store_row<G, SB>(p.lv.snaps, d_off + static_cast<size_t>(r + m * G::kPer) * DK, s[m]);
        }
        __syncthreads();  // this buffer is refilled by the next pass
    }
#pragma unroll
    for (int m = 0; m < kRows; ++m) store_row<G, SB>(p.lv.states, s_off + static_cast<size_t>(r + m * G::kPer) * DK, s[m]);
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
    auto kernel = gdn_run_kernel<DK, SB, IB, false>;
    if constexpr (SB)
        if (!a.cu_seqlens) kernel = gdn_run_kernel<DK, SB, IB, true>;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(32 * warps), 0, s, a, tiles);
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
