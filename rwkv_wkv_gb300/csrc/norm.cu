// The gated norm of a layer's readout: over groups of columns of each row
//     y = (u - m) r w + b,   m = 0, r = (mean u^2 + eps)^-1/2            (rms)
//                            m = mean u, r = (mean (u - m)^2 + eps)^-1/2  (layer)
// of u = x act(z) (the gate first) or of u = x, the result then multiplied by act(z).
//
// One pass: a group's values stay in registers, eight neighbouring columns a thread, between
// its sum and its outputs; every sum is float32 in a fixed order, deviations from the mean are taken
// before they are squared.  Groups of up to 256 columns lie in the lanes of one warp, which takes
// several at a time so that their loads overlap; longer ones have a CTA each.  Bound by HBM.
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

__device__ __forceinline__ float gate_of(int act, float z) {
    return act == WKV7_GATE_SILU ? silu(z) : act == WKV7_GATE_SIGMOID ? sigmoid(z) : z;
}

// Sum over `lanes` neighbouring lanes (a power of two); every lane gets it.
__device__ __forceinline__ float sum_over(float x, int lanes) {
    for (int off = 1; off < lanes; off *= 2) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

__device__ __forceinline__ float square_sum(const float (&x)[kVec]) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kVec; ++e) s = fmaf(x[e], x[e], s);
    return s;
}

// x as the norm sees it, and what its result is multiplied by (with the gate last).
template <bool XB, bool ZB>
struct Cells {
    float x[kVec], z[kVec];
    __device__ __forceinline__ void load(const wkv7_norm_args &p, long long row, int col) {
        load8<XB>(p.x, static_cast<size_t>(row * p.x_stride + col), x);
        if (p.z) load8<ZB>(p.z, static_cast<size_t>(row * p.z_stride + col), z);
    }
    __device__ __forceinline__ void gate_first(const wkv7_norm_args &p) {
        if (p.z && p.gate_first) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[e] *= gate_of(p.act, z[e]);
        }
    }
    // y of columns col .. col + 7, from u - m in x and r
    __device__ __forceinline__ void store(const wkv7_norm_args &p, long long row, int col, float r) {
        float w[kVec], b[kVec];
        if (p.weight) {
            if (p.w_dtype == WKV7_BF16) load8<true>(p.weight, col, w);
            else load8<false>(p.weight, col, w);
        }
        if (p.bias) {
            if (p.w_dtype == WKV7_BF16) load8<true>(p.bias, col, b);
            else load8<false>(p.bias, col, b);
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            float y = x[e] * r;
            if (p.weight) y *= w[e];
            if (p.bias) y += b[e];
            x[e] = p.z && !p.gate_first ? y * gate_of(p.act, z[e]) : y;
        }
        const size_t at = static_cast<size_t>(row) * p.width + col;
        if (p.o_dtype == WKV7_BF16) store8<true>(p.o, at, x);
        else store8<false>(p.o, at, x);
    }
};

// Groups in the lanes of a warp: `lanes` (a power of two) of them hold a group, kTurns groups each.
constexpr int kTurns = 4;

template <bool XB, bool ZB>
__global__ void __launch_bounds__(256) norm_small_kernel(const wkv7_norm_args p, int lanes, long long groups, int per_row) {
    pdl_prologue();
    const int vecs = p.group / kVec, lane = threadIdx.x & 31;
    const int at = lane & (lanes - 1), per_warp = 32 / lanes;
    const long long warp = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const long long first = warp * (kTurns * per_warp) + lane / lanes;
    const float share = 1.f / static_cast<float>(p.group);
    Cells<XB, ZB> c[kTurns];
    long long row[kTurns];
    int col[kTurns];
    bool live[kTurns];
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        const long long g = first + t * per_warp;
        live[t] = g < groups && at < vecs;
        row[t] = g / per_row;
        col[t] = static_cast<int>(g - row[t] * per_row) * p.group + at * kVec;
        if (live[t]) {
            c[t].load(p, row[t], col[t]);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) c[t].x[e] = 0.f, c[t].z[e] = 0.f;
        }
    }
#pragma unroll
    for (int t = 0; t < kTurns; ++t) {
        c[t].gate_first(p);
        if (p.kind == WKV7_NORM_LAYER) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < kVec; ++e) s += c[t].x[e];
            s = sum_over(s, lanes) * share;
#pragma unroll
            for (int e = 0; e < kVec; ++e) c[t].x[e] = at < vecs ? c[t].x[e] - s : 0.f;
        }
        const float r = rsqrtf(fmaf(sum_over(square_sum(c[t].x), lanes), share, p.eps));
        if (live[t]) c[t].store(p, row[t], col[t], r);
    }
}

// Sum over the CTA in a fixed order; every thread gets it.
__device__ __forceinline__ float sum_cta(float x, float *part) {
    x = sum_over(x, 32);
    const int warps = blockDim.x >> 5;
    __syncthreads();  // an earlier sum's parts are read
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return sum_over(lane < warps ? part[lane] : 0.f, 32);
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
        const int v = threadIdx.x + i * blockDim.x;
        if (v < vecs) {
            c[i].load(p, row, col0 + v * kVec);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e) c[i].x[e] = 0.f, c[i].z[e] = 0.f;
        }
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        c[i].gate_first(p);
        if (p.kind == WKV7_NORM_LAYER) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) s += c[i].x[e];
        }
    }
    if (p.kind == WKV7_NORM_LAYER) {
        s = sum_cta(s, part) * share;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < kVec; ++e) c[i].x[e] = threadIdx.x + i * blockDim.x < vecs ? c[i].x[e] - s : 0.f;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) q += square_sum(c[i].x);
    const float r = rsqrtf(fmaf(sum_cta(q, part), share, p.eps));
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < vecs) c[i].store(p, row, col0 + v * kVec, r);
    }
}

template <bool XB, bool ZB>
cudaError_t norm_as(const wkv7_norm_args &a, cudaStream_t s) {
    const int vecs = a.group / kVec, per_row = a.width / a.group;
    const long long groups = static_cast<long long>(a.rows) * per_row;
    if (vecs <= 32) {
        int lanes = 1;
        while (lanes < vecs) lanes *= 2;
        const long long per_cta = 8LL * kTurns * (32 / lanes);
        const long long ctas = (groups + per_cta - 1) / per_cta;
        if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
        return launch_pdl(norm_small_kernel<XB, ZB>, dim3(static_cast<unsigned>(ctas)), dim3(256), 0, s, a, lanes, groups, per_row);
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
