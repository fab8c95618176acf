// The short causal convolution over the tokens of a request, a filter per channel:
//     o_t = act(bias + sum_{j < W} w[j] u_{t - W + 1 + j}),   act(x) = x / (1 + e^-x) or x.
// What lies before a call's first token comes from the request's slot, which keeps the last
// W - 1 inputs as they came, [W - 1][channels], oldest first; the newest go back there.
//
// A thread takes four neighbouring channels, 8 bytes of a bf16 row, and walks along the tokens with
// the last W - 1 inputs in registers, so that each input is loaded and widened once (and W - 1 of
// them again at a tile's start).  Sums are float32, a fused multiply-add a tap.  The bytes of x and o bound it,
// and the SiLU's two approximate functions a value are not far behind: 33.6 thousand tokens of 64 ragged prompts, 4,096
// channels of bf16, 0.55 GB, 108 us (5.1 TB/s, 77% of the copy rate); 119 where the next rows are not on their way
// while these are worked on, 148 with eight channels a thread (twice the registers, half of the loads on their way).
// Short calls are bound by the launch: 256 rows of 4,352 channels and their tails 4.2 us.
#include "device_common.cuh"
#include "gate.cuh"
#include "packed_f32.cuh"
#include "ssm_internal.h"

namespace wkv7 {
namespace {

constexpr int kVec = kConvVec;  // channels a thread
constexpr int kAhead = 4;  // rows of a sequence loaded at a time

// Four inputs as they come: of bf16, or of float32.
template <bool BF>
struct RawOf {
    using Type = uint2;
};
template <>
struct RawOf<false> {
    using Type = uint4;
};
template <bool BF>
using Raw = typename RawOf<BF>::Type;
template <bool BF>
__device__ __forceinline__ const Raw<BF> *raw_at(const void *p, size_t off) {
    return reinterpret_cast<const Raw<BF> *>(static_cast<const char *>(p) + off * (BF ? 2 : 4));
}
template <bool BF>
__device__ __forceinline__ Raw<BF> load_raw(const void *p, size_t off) {
    return *raw_at<BF>(p, off);
}
// As load_raw, of values that the kernel does not write.
template <bool BF>
__device__ __forceinline__ Raw<BF> load_row(const void *p, size_t off) {
    return __ldg(raw_at<BF>(p, off));
}
template <bool BF>
__device__ __forceinline__ void store_raw(void *p, size_t off, const Raw<BF> &r) {
    *const_cast<Raw<BF> *>(raw_at<BF>(p, off)) = r;
}
// As pairs of floats.
struct Four {
    F2 v[2];
};
__device__ __forceinline__ Four widen(uint2 r) { return {{f2_bf16(r.x), f2_bf16(r.y)}}; }
__device__ __forceinline__ Four widen(uint4 r) {
    return {{f2(__uint_as_float(r.x), __uint_as_float(r.y)), f2(__uint_as_float(r.z), __uint_as_float(r.w))}};
}

// A thread's filters, taps first, and bias.
template <int W>
struct Filter {
    Four w[W], bias;
};
template <int W, bool WB>
__device__ __forceinline__ Filter<W> load_filter_as(const ConvArgs &p, int ch) {
    Filter<W> f;
    float x[kVec * W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float4 u = load4<WB>(p.weight, static_cast<size_t>(ch) * W + 4 * i);
        x[4 * i] = u.x, x[4 * i + 1] = u.y, x[4 * i + 2] = u.z, x[4 * i + 3] = u.w;
    }
#pragma unroll
    for (int j = 0; j < W; ++j) f.w[j] = {{f2(x[j], x[W + j]), f2(x[2 * W + j], x[3 * W + j])}};
    const float4 b = p.bias ? load4<WB>(p.bias, ch) : make_float4(0.f, 0.f, 0.f, 0.f);
    f.bias = {{f2(b.x, b.y), f2(b.z, b.w)}};
    return f;
}
template <int W>
__device__ __forceinline__ Filter<W> load_filter(const ConvArgs &p, int ch) {
    return p.w_bf16 ? load_filter_as<W, true>(p, ch) : load_filter_as<W, false>(p, ch);
}

// One output of each channel from the last W inputs, oldest first.
template <int W, bool BF>
__device__ __forceinline__ void emit(const ConvArgs &p, const Filter<W> &f, const Four (&u)[W], size_t at) {
    F2 acc[2] = {f.bias.v[0], f.bias.v[1]};
#pragma unroll
    for (int j = 0; j < W; ++j) {
        acc[0] = fma2(u[j].v[0], f.w[j].v[0], acc[0]);
        acc[1] = fma2(u[j].v[1], f.w[j].v[1], acc[1]);
    }
    float x[kVec];
    unpack(acc[0], x[0], x[1]);
    unpack(acc[1], x[2], x[3]);
    if (p.silu) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[e] = silu(x[e]);
    }
    if constexpr (BF)
        store_raw<true>(p.o, at, make_uint2(pack_bf16_rn(x[0], x[1]), pack_bf16_rn(x[2], x[3])));
    else
        store_raw<false>(p.o, at, make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])));
}

template <bool BF>
__device__ __forceinline__ size_t tail_at(const ConvArgs &p, int id, int j, int ch) {  // in elements
    return (static_cast<size_t>(id) * p.slot_bytes + p.layer_off) / (BF ? 2 : 4) + static_cast<size_t>(j) * p.channels + ch;
}

// ---------------------------------------------------------- tokens of many slots

// n_tok tokens of each of n slots; with step_snap_ids the tail after each token also goes to its snapshot.
template <int W, bool BF>
__global__ void __launch_bounds__(128) conv_step_kernel(const ConvArgs p) {
    pdl_prologue();
    const int ch = (blockIdx.x * blockDim.x + threadIdx.x) * kVec;
    const int bi = blockIdx.y + blockIdx.z * 65535;
    if (ch >= p.channels || bi >= p.n) return;
    const int slot = __ldg(p.slot_ids + bi);
    if (slot < 0 || slot >= p.n_slots) {
        if (ch == 0) flag_status(p.status, WKV7_DEV_BAD_SLOT);
        return;
    }
    const long long row0 = static_cast<long long>(bi) * p.n_tok;
    Raw<BF> u[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) u[j] = load_raw<BF>(p.slots, tail_at<BF>(p, slot, j, ch));
    u[W - 1] = load_raw<BF>(p.x, static_cast<size_t>(row0 * p.x_stride + ch));
    const Filter<W> f = load_filter<W>(p, ch);
    for (int t = 0; t < p.n_tok; ++t) {
        Raw<BF> next = u[W - 1];
        if (t + 1 < p.n_tok) next = load_raw<BF>(p.x, static_cast<size_t>((row0 + t + 1) * p.x_stride + ch));
        Four w[W];
#pragma unroll
        for (int j = 0; j < W; ++j) w[j] = widen(u[j]);
        emit<W, BF>(p, f, w, static_cast<size_t>(row0 + t) * p.channels + ch);
        if (p.step_snap_ids) {
            const int id = __ldg(p.step_snap_ids + row0 + t);
            if (id >= 0 && id < p.n_snaps) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) store_raw<BF>(p.snaps, tail_at<BF>(p, id, j, ch), u[j + 1]);
            } else if (ch == 0) {
                flag_status(p.status, WKV7_DEV_BAD_SLOT);
            }
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) u[j] = u[j + 1];
        u[W - 1] = next;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_raw<BF>(p.slots, tail_at<BF>(p, slot, j, ch), u[j]);
}

// ------------------------------------------------------------------- sequences

// One CTA walks T packed tokens for its channels.  Every CTA reads all of cu_seqlens, to find which
// sequences its tokens belong to and whether the array is consistent; if not, nothing is written.
//
// A sequence's first W - 1 tokens need its old tail, which the new one replaces.  All of them are
// computed by the CTA whose tile holds the first one, also those past its tile's end, and the
// same thread then stores the new tail: so only one thread ever reads the old values.
template <int W, bool BF, int T>
__global__ void __launch_bounds__(128) conv_prefill_kernel(const ConvArgs p) {
    __shared__ int seq_of[T + W - 1];  // of this CTA's tokens; -1: another CTA's, or no sequence's
    const int tid = threadIdx.x;
    for (int i = tid; i < T + W - 1; i += blockDim.x) seq_of[i] = -1;  // (a CTA may have fewer threads than that)
    pdl_prologue();
    __syncthreads();
    const int t0 = blockIdx.x * T, t1 = min(t0 + T, p.total_tokens);
    bool bad = false;
    for (int s = tid; s < p.n; s += blockDim.x) {
        const int a = __ldg(p.cu_seqlens + s), b = __ldg(p.cu_seqlens + s + 1);
        if (a < 0 || b < a || b > p.total_tokens) {
            bad = true;
        } else if (b > t0 && a < t1) {
            const int from = a >= t0 ? a : max(t0, static_cast<int>(min(static_cast<long long>(a) + W - 1, static_cast<long long>(b))));
            const int to = min(b, a >= t0 ? max(t1, a + W - 1) : t1);
            for (int t = from; t < to; ++t) seq_of[t - t0] = s;  // (disjoint where the array is consistent)
        }
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) flag_status(p.status, WKV7_DEV_BAD_SEQLENS);
        return;
    }
    const int ch = (blockIdx.y * blockDim.x + tid) * kVec;
    if (ch >= p.channels) return;
    const Filter<W> f = load_filter<W>(p, ch);
    auto row = [&](int t) { return load_row<BF>(p.x, static_cast<size_t>(t * p.x_stride + ch)); };
    int cur = -1;
    bool skip = false;
    Four u[W];
    const int end = min(t1 - t0 + W - 1, p.total_tokens - t0);
    // the next rows are on their way while these are worked on
    auto rows_at = [&](int i0, Raw<BF> (&in)[kAhead]) {
        if (i0 + kAhead <= end) {
            size_t at = static_cast<size_t>((t0 + i0) * p.x_stride + ch);
#pragma unroll
            for (int k = 0; k < kAhead; ++k, at += p.x_stride) in[k] = load_row<BF>(p.x, at);
        } else {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) in[k] = row(min(t0 + i0 + k, t0 + end - 1));
        }
    };
    Raw<BF> in[kAhead], next[kAhead];
    rows_at(0, next);
    for (int i0 = 0; i0 < end; i0 += kAhead) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) in[k] = next[k];
        if (i0 + kAhead < end) rows_at(i0 + kAhead, next);
        // (the branches are the same for the whole CTA)
        if (!skip && i0 + kAhead <= end && seq_of[i0] == cur && cur >= 0 && seq_of[i0 + kAhead - 1] == cur) {
            size_t at = static_cast<size_t>(t0 + i0) * p.channels + ch;
#pragma unroll
            for (int k = 0; k < kAhead; ++k, at += p.channels) {
                u[W - 1] = widen(in[k]);
                emit<W, BF>(p, f, u, at);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) u[j] = u[j + 1];
            }
            continue;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k, t = t0 + i;
            const int s = i < end ? seq_of[i] : -1;
            if (s < 0) continue;
            if (s != cur) {
                cur = s;
                const int a = __ldg(p.cu_seqlens + s), b = __ldg(p.cu_seqlens + s + 1);
                const int slot = __ldg(p.slot_ids + s);
                skip = slot < 0 || slot >= p.n_slots;
                if (skip) {
                    if (tid == 0 && blockIdx.y == 0) flag_status(p.status, WKV7_DEV_BAD_SLOT);
                    continue;
                }
                if (t == a) {
                    Raw<BF> old[W - 1];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) old[j] = load_raw<BF>(p.slots, tail_at<BF>(p, slot, j, ch));
                    const int len = b - a;
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {  // the last W - 1 of (old tail, tokens)
                        const int from = len + j;
                        Raw<BF> newest = old[0];
#pragma unroll
                        for (int m = 1; m < W - 1; ++m)
                            if (from == m) newest = old[m];
                        if (from >= W - 1) newest = row(a + from - (W - 1));
                        store_raw<BF>(p.slots, tail_at<BF>(p, slot, j, ch), newest);
                    }
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) u[j] = widen(old[j]);
                } else {  // W - 1 tokens of it lie before this one
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) u[j] = widen(row(t - (W - 1) + j));
                }
            }
            if (skip) continue;
            u[W - 1] = widen(in[k]);
            emit<W, BF>(p, f, u, static_cast<size_t>(t) * p.channels + ch);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) u[j] = u[j + 1];
        }
    }
}

template <int W, bool BF>
cudaError_t step_as(const ConvArgs &a, cudaStream_t s) {
    const unsigned x = static_cast<unsigned>((a.channels / kVec + 127) / 128), n = static_cast<unsigned>(a.n);
    return launch_pdl(conv_step_kernel<W, BF>, dim3(x, n < 65535u ? n : 65535u, (n + 65534u) / 65535u), dim3(128), 0, s, a);
}

template <int W, bool BF>
cudaError_t prefill_as(const ConvArgs &a, cudaStream_t s) {
    const ConvTiles t = conv_tiles(a.channels, a.total_tokens);
    auto kernel = t.tokens == 64 ? conv_prefill_kernel<W, BF, 64>
                                 : t.tokens == 32 ? conv_prefill_kernel<W, BF, 32> : conv_prefill_kernel<W, BF, 8>;
    return launch_pdl(kernel, dim3(t.tiles, t.blocks), dim3(t.threads), 0, s, a);
}

}  // namespace

cudaError_t launch_conv_step(const ConvArgs &a, cudaStream_t s, int *launches) {
    cudaError_t (*const as[6])(const ConvArgs &, cudaStream_t) = {step_as<2, false>, step_as<2, true>, step_as<3, false>,
                                                                  step_as<3, true>,  step_as<4, false>, step_as<4, true>};
    const cudaError_t e = as[(a.width - 2) * 2 + (a.bf16 ? 1 : 0)](a, s);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_conv_prefill(const ConvArgs &a, cudaStream_t s, int *launches) {
    cudaError_t (*const as[6])(const ConvArgs &, cudaStream_t) = {prefill_as<2, false>, prefill_as<2, true>, prefill_as<3, false>,
                                                                  prefill_as<3, true>,  prefill_as<4, false>, prefill_as<4, true>};
    const cudaError_t e = as[(a.width - 2) * 2 + (a.bf16 ? 1 : 0)](a, s);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace wkv7
