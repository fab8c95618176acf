// The gated norm of a layer's readout: over groups of columns of each row
//     y = (u - m) r w + b,   m = 0, r = (mean u^2 + eps)^-1/2            (rms)
//                            m = mean u, r = (mean (u - m)^2 + eps)^-1/2  (layer)
// of u = x act(z) (the gate first) or of u = x, the result then multiplied by act(z).
//
// One pass: a group's values stay in registers, eight neighbouring columns a thread, between
// its sum and its outputs; every sum is float32 in a fixed order, deviations from the mean are taken
// before they are squared.  Groups of up to 256 columns lie in the lanes of one warp, which takes
// several at a time so that their loads overlap; longer ones have a CTA each.  Bound by HBM, and for few
// rows by the launch: 256 rows of 4,096, the norm over all of a row, 3.5 us.
#include "device_common.cuh"
#include "gate.cuh"
#include "ssm_internal.h"

namespace wkv7 {
namespace {

constexpr int kVec = 8;

template <bool BF>
__device__ __forceinline__ void store8(void *o, size_t off, const float (&x)[kVec]) {
    if constexpr (BF) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(o) + off) =
            make_uint4(pack_bf16_rn(x[0], x[1]), pack_bf16_rn(x[2], x[3]), pack_bf16_rn(x[4], x[5]), pack_bf16_rn(x[6], x[7]));
    } else {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(o) + off);
        q[0] = make_float4(x[0], x[1], x[2], x[3]);
        q[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// Sum over LANES neighbouring lanes (a power of two); every lane gets it.
template <int LANES>
__device__ __forceinline__ float sum_over(float x) {
#pragma unroll
    for (int off = 1; off < LANES; off *= 2) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

__device__ __forceinline__ float square_sum(const float (&x)[kVec]) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kVec; ++e) s = fmaf(x[e], x[e], s);
    return s;
}

// Eight values as they come.
template <bool BF>
struct Raw {
    uint4 u[BF ? 1 : 2];
    __device__ __forceinline__ void load(const void *p, size_t off) {
        const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const char *>(p) + off * (BF ? 2 : 4));
        u[0] = __ldcs(q);
        if (!BF) u[BF ? 0 : 1] = __ldcs(q + 1);
    }
    __device__ __forceinline__ void zero() { u[0] = u[BF ? 0 : 1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void widen(float (&x)[kVec]) const {
        const uint32_t a[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
        if constexpr (BF) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(a[i]), x[2 * i + 1] = bf16_hi(a[i]);
        } else {
            const uint32_t b[4] = {u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(a[i]), x[4 + i] = __uint_as_float(b[i]);
        }
    }
};

// x as the norm sees it, and the gate as it came.
template <bool XB, bool ZB>
struct Cells {
    Raw<XB> x;
    Raw<ZB> z;
    __device__ __forceinline__ void load(const wkv7_norm_args &p, long long row, int col) {
        x.load(p.x, static_cast<size_t>(row * p.x_stride + col));
        if (p.z) z.load(p.z, static_cast<size_t>(row * p.z_stride + col));
    }
    __device__ __forceinline__ void zero() { x.zero(), z.zero(); }
    __device__ __forceinline__ void values(const wkv7_norm_args &p, float (&v)[kVec]) const {
        x.widen(v);
        if (p.z && p.gate_first) gate(p, v);
    }
    __device__ __forceinline__ void gate(const wkv7_norm_args &p, float (&v)[kVec]) const {
        float g[kVec];
        z.widen(g);
        if (p.act == WKV7_GATE_SILU) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[e] *= silu(g[e]);  // (the gate first: v g alone may overflow)
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[e] *= p.act == WKV7_GATE_SIGMOID ? sigmoid(g[e]) : g[e];
        }
    }
    // y of columns col .. col + 7, from u - m in v and r
    __device__ __forceinline__ void store(const wkv7_norm_args &p, long long row, int col, float (&v)[kVec], float r) const {
        float w[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] *= r;
        if (p.weight) {
            if (p.w_dtype == WKV7_BF16) load8<true>(p.weight, col, w);
            else load8<false>(p.weight, col, w);
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[e] *= w[e];
        }
        if (p.bias) {
            if (p.w_dtype == WKV7_BF16) load8<true>(p.bias, col, w);
            else load8<false>(p.bias, col, w);
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[e] += w[e];
        }
        if (p.z && !p.gate_first) gate(p, v);
        const size_t at = static_cast<size_t>(row) * p.width + col;
        if (p.o_dtype == WKV7_BF16) store8<true>(p.o, at, v);
        else store8<false>(p.o, at, v);
    }
};

// Groups in the lanes of a warp: LANES of them hold a group, a few groups each.  What a thread
// holds between its loads and its outputs stays as it came, and is kept to 64 registers (8 bytes spilled where x and z are
// bf16), so that 32 warps fit an SM: 32,768 rows of 32 groups of 128, bf16, 134 us (6.0 TB/s), 151 with 72 registers, 362
// with floats held.
template <bool XB, bool ZB>
constexpr int kTurnsOf = XB && ZB ? 4 : 2;

template <bool XB, bool ZB, int LANES>
__global__ void __launch_bounds__(256, 4) norm_small_kernel(const wkv7_norm_args p, long long groups, int per_row) {
    pdl_prologue();
    constexpr int kPerWarp = 32 / LANES, kTurns = kTurnsOf<XB, ZB>;
    const int vecs = p.group / kVec, lane = threadIdx.x & 31, at = lane & (LANES - 1);
    // the CTA's first group's row, and from there on in 32 bits (a division of 64 is as long as the rest)
    const long long first = static_cast<long long>(blockIdx.x) * (8 * kTurns * kPerWarp);
    const long long row0 = groups <= 0xffffffffLL ? static_cast<unsigned>(first) / static_cast<unsigned>(per_row) : first / per_row;
    const int col0 = static_cast<int>(first - row0 * per_row) + (threadIdx.x >> 5) * (kTurns * kPerWarp) + lane / LANES;
    const float share = 1.f / static_cast<float>(p.group);
    Cells<XB, ZB> c[kTurns];
    long long row[kTurns];
    int col[kTurns];
    bool live[kTurns];
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        const unsigned g = static_cast<unsigned>(col0 + t * kPerWarp), down = g / static_cast<unsigned>(per_row);
        row[t] = row0 + down;
        col[t] = static_cast<int>(g - down * per_row) * p.group + at * kVec;
        live[t] = row[t] < p.rows && at < vecs;
        if (live[t]) c[t].load(p, row[t], col[t]);
        else c[t].zero();
    }
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        float v[kVec];
        c[t].values(p, v);
        if (p.kind == WKV7_NORM_LAYER) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < kVec; ++e) s += v[e];
            s = sum_over<LANES>(s) * share;
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[e] = at < vecs ? v[e] - s : 0.f;
        }
        const float r = rsqrtf(fmaf(sum_over<LANES>(square_sum(v)), share, p.eps));
        if (live[t]) c[t].store(p, row[t], col[t], v, r);
    }
}

// Sum over the CTA in a fixed order; every thread gets it.
__device__ __forceinline__ float sum_cta(float x, float *part) {
    x = sum_over<32>(x);
    const int warps = blockDim.x >> 5;
    __syncthreads();  // an earlier sum's parts are read
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return sum_over<32>(lane < warps ? part[lane] : 0.f);
}

// A group in a CTA, R times eight columns a thread.
constexpr int R = 2;

template <bool XB, bool ZB>
__global__ void __launch_bounds__(1024) norm_large_kernel(const wkv7_norm_args p, int per_row) {
    __shared__ float part[32];
    pdl_prologue();
    const long long row = blockIdx.x / per_row;
    const int col0 = static_cast<int>(blockIdx.x % per_row) * p.group, vecs = p.group / kVec;
    const float share = 1.f / static_cast<float>(p.group);
    Cells<XB, ZB> c[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int at = threadIdx.x + i * blockDim.x;
        if (at < vecs) c[i].load(p, row, col0 + at * kVec);
        else c[i].zero();
    }
    float v[R][kVec];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        c[i].values(p, v[i]);
        if (p.kind == WKV7_NORM_LAYER) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) s += v[i][e];
        }
    }
    if (p.kind == WKV7_NORM_LAYER) {
        s = sum_cta(s, part) * share;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[i][e] = threadIdx.x + i * blockDim.x < vecs ? v[i][e] - s : 0.f;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) q += square_sum(v[i]);
    const float r = rsqrtf(fmaf(sum_cta(q, part), share, p.eps));
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int at = threadIdx.x + i * blockDim.x;
        if (at < vecs) c[i].store(p, row, col0 + at * kVec, v[i], r);
    }
}

template <bool XB, bool ZB>
cudaError_t norm_as(const wkv7_norm_args &a, cudaStream_t s) {
    const int vecs = a.group / kVec, per_row = a.width / a.group;
    const long long groups = static_cast<long long>(a.rows) * per_row;
    if (vecs <= 32) {
        int lanes = 1, pick = 0;
        while (lanes < vecs) lanes *= 2, ++pick;
        const long long per_cta = 8LL * kTurnsOf<XB, ZB> * (32 / lanes);
        const long long ctas = (groups + per_cta - 1) / per_cta;
        if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
        void (*const as[6])(wkv7_norm_args, long long, int) = {norm_small_kernel<XB, ZB, 1>, norm_small_kernel<XB, ZB, 2>,
                                                               norm_small_kernel<XB, ZB, 4>, norm_small_kernel<XB, ZB, 8>,
                                                               norm_small_kernel<XB, ZB, 16>, norm_small_kernel<XB, ZB, 32>};
        return launch_pdl(as[pick], dim3(static_cast<unsigned>(ctas)), dim3(256), 0, s, a, groups, per_row);
    }
    if (groups > 0x7fffffffLL) return cudaErrorInvalidValue;
    const int threads = ((vecs + R - 1) / R + 31) / 32 * 32;  // at most 1024: groups of 16,384
    return launch_pdl(norm_large_kernel<XB, ZB>, dim3(static_cast<unsigned>(groups)), dim3(static_cast<unsigned>(threads)), 0, s, a, per_row);
}

}  // namespace

cudaError_t launch_gated_norm(const wkv7_norm_args &a, cudaStream_t s, int *launches) {
    const bool xb = a.x_dtype == WKV7_BF16, zb = a.z_dtype == WKV7_BF16;
    const cudaError_t e = xb ? (zb ? norm_as<true, true>(a, s) : norm_as<true, false>(a, s))
                             : (zb ? norm_as<false, true>(a, s) : norm_as<false, false>(a, s));
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace wkv7
