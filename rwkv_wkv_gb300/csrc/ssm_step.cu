// The selective scan token by token: single-token decode over indirected state
// slots, and runs of tokens (multi-token decode with rollback states, prefill in
// float32).
//
// Per head (S[i][j]: i of p, j of d_state) every token does
//     S <- a S + (dt x) B^T,  a = exp(dt A);   o = S C + D x.
// Row i of S needs only itself, B, C and x_i, so any set of rows is a unit of work: a warp
// holds kRows of them per lane group in registers, 16 bytes of a row per lane, and the
// readouts of its rows are summed over the lanes by one reduce-scatter.
//
// Decode is bound by HBM: a 64 x 128 float32 head moves 64 KiB for 41 kFLOP.  256 slots of 64 such heads, 1.08 GB,
// take 156 us (6.9 TB/s, the copy rate); one slot 2.3 us, the launch and three dependent reads; 203 slots of 24 heads of
// 64 x 64, bf16 states and float32 inputs, 82 MB that stay in L2, 11.9 us.  A run with a state to keep after each token is
// bound by writing them: 48 slots x 5 tokens x 32 heads, 0.36 GB, 55 us (6.5 TB/s).  Long runs are bound by their
// instructions and the inputs' staging: 0.25 us a token where few heads run, 8 x 4,096 tokens of 64 heads 4.7 ms.
//
// Every product and sum of the state's update is written out: K tokens of a run leave the bits of
// K single steps.  With bf16 states the update is rounded as the formula is written (a S, dt x and
// its product with B each to float32, then their sum), so that whoever evaluates it so in float32
// has the stored bits.
#include "device_common.cuh"
#include "ssm_internal.h"
#include "ssm_scalars.cuh"

#include <type_traits>

namespace wkv7 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kFirstWaveCtas = 152 * 16;  // CTAs that may start while the previous kernel drains

// How a warp covers rows of N state entries.
template <int N, bool SB>
struct Geo {
    static constexpr int kCols = SB ? 8 : 4;            // entries per lane
    static constexpr int kRows = SB ? 4 : 8;            // rows per lane group
    static constexpr int kLanes = N / kCols;            // lanes per row
    static constexpr int kPer = 32 / kLanes;            // rows per warp access
    static constexpr int kWarpRows = kPer * kRows;
    static constexpr int kTile = kWarps * kWarpRows;    // rows per CTA: 32 or 64
    static constexpr int kRest = kLanes / kRows;        // lanes that end with the same row's sum
    // the row (of its group's kRows) whose sum a lane ends with, and whether it is the one that stores it
    static __device__ __forceinline__ int own_row(int lane) { return (lane & (kLanes - 1)) / kRest; }
    static __device__ __forceinline__ bool owns(int lane) { return (lane & (kRest - 1)) == 0; }
};

template <class G, bool SB>
__device__ __forceinline__ void load_row(const float *base, size_t off, float (&x)[G::kCols]) {
    if constexpr (SB) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(base) + off));
        x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
        x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
    } else {
        const float4 u = __ldcs(reinterpret_cast<const float4 *>(base + off));
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    }
}
template <class G, bool SB>
__device__ __forceinline__ void store_row(float *base, size_t off, const float (&x)[G::kCols]) {
    if constexpr (SB)
        __stcs(reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(base) + off),
               make_uint4(pack_bf16_rn(x[0], x[1]), pack_bf16_rn(x[2], x[3]), pack_bf16_rn(x[4], x[5]), pack_bf16_rn(x[6], x[7])));
    else
        __stcs(reinterpret_cast<float4 *>(base + off), make_float4(x[0], x[1], x[2], x[3]));
}

// kCols entries of B or C (global or shared memory) as floats.
template <class G, bool IB>
__device__ __forceinline__ void load_in(const void *p, size_t off, float (&x)[G::kCols]) {
    if constexpr (IB && G::kCols == 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + off);
        x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
        x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
    } else if constexpr (IB) {
        const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + off);
        x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
    } else {
#pragma unroll
        for (int c = 0; c < G::kCols; c += 4) {
            const float4 u = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + off + c);
            x[c] = u.x; x[c + 1] = u.y; x[c + 2] = u.z; x[c + 3] = u.w;
        }
    }
}

// One token on the rows a lane holds; returns the readout S C of row own_row(lane).
template <class G, bool SB>
__device__ __forceinline__ float token_step(float (&s)[G::kRows][G::kCols], const float (&b)[G::kCols],
                                            const float (&c)[G::kCols], const float (&x)[G::kRows], const StepScalars &t,
                                            int lane) {
    float v[G::kRows];
#pragma unroll
    for (int m = 0; m < G::kRows; ++m) {
        const float u = __fmul_rn(t.dt, x[m]);
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < G::kCols; ++e) {
            const float add = __fmul_rn(u, b[e]);
            s[m][e] = SB ? __fadd_rn(__fmul_rn(t.a, s[m][e]), add) : __fmaf_rn(t.a, s[m][e], add);
            sum = __fmaf_rn(s[m][e], c[e], sum);
        }
        v[m] = sum;
    }
    int off = G::kLanes / 2;
#pragma unroll
    for (int n = G::kRows; n > 1; n /= 2, off /= 2) {
        const bool hi = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = hi ? v[i + n / 2] : v[i];
            const float send = hi ? v[i] : v[i + n / 2];
            v[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, send, off));
        }
    }
#pragma unroll
    for (; off >= 1; off /= 2) v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xffffffffu, v[0], off));
    return v[0];
}

// ------------------------------------------------------------------- decode

// One CTA advances kTile rows of one (batch row, head).  It reads its slot id and warms L2
// with its rows before it waits for the previous kernel, as the other pools' decode does.
template <int N, bool SB, bool IB>
__global__ void __launch_bounds__(kThreads) ssm_decode_kernel(const SsmRunArgs p, int tiles) {
    using G = Geo<N, SB>;
    pdl_launch_dependents();
    const int unit = blockIdx.x / tiles, tile = blockIdx.x - unit * tiles;
    const int bi = unit / p.lv.heads, h = unit - bi * p.lv.heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = tile * G::kTile + warp * G::kWarpRows;  // this warp's first row
    const int r = row0 + lane / G::kLanes;                   // this lane's first row
    const int c0 = (lane & (G::kLanes - 1)) * G::kCols;
    const int slot = __ldg(p.slot_ids + bi);
    const bool ok = slot >= 0 && slot < p.lv.n_slots;
    const size_t s_off = static_cast<size_t>(ok ? slot : 0) * p.lv.slot_stride + p.lv.layer_off +
                         static_cast<size_t>(h) * p.lv.p * N + c0;
    if (ok && blockIdx.x < kFirstWaveCtas && (lane & 7) == 0) {  // one prefetch per 128-byte line
#pragma unroll
        for (int m = 0; m < G::kRows; ++m) {
            const size_t off = s_off + static_cast<size_t>(r + m * G::kPer) * N;
            prefetch_l2(SB ? static_cast<const void *>(reinterpret_cast<const uint16_t *>(p.lv.states) + off)
                           : static_cast<const void *>(p.lv.states + off));
        }
    }
    pdl_wait();
    if (!ok) {
        if (threadIdx.x == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SLOT);
        return;
    }
    float s[G::kRows][G::kCols];
#pragma unroll
    for (int m = 0; m < G::kRows; ++m) load_row<G, SB>(p.lv.states, s_off + static_cast<size_t>(r + m * G::kPer) * N, s[m]);
    const int g = h / (p.lv.heads / p.lv.groups);
    const float dt = load_dt(p.in, bi, h);
    float b[G::kCols], c[G::kCols], x[G::kRows];
    load_in<G, IB>(p.in.b, static_cast<size_t>(bi) * p.in.b_stride + static_cast<size_t>(g) * N + c0, b);
    load_in<G, IB>(p.in.c, static_cast<size_t>(bi) * p.in.c_stride + static_cast<size_t>(g) * N + c0, c);
    const size_t x_off = static_cast<size_t>(bi) * p.in.x_stride + static_cast<size_t>(h) * p.lv.p;
#pragma unroll
    for (int m = 0; m < G::kRows; ++m) x[m] = load1<IB>(p.in.x, x_off + r + m * G::kPer);
    const int mine = r + G::own_row(lane) * G::kPer;
    const float x_own = load1<IB>(p.in.x, x_off + mine);
    const float d = p.in.d ? __ldg(p.in.d + h) : 0.f;
    const StepScalars t = step_scalars(p.in, h, dt);
    const float y = token_step<G, SB>(s, b, c, x, t, lane);
#pragma unroll
    for (int m = 0; m < G::kRows; ++m) store_row<G, SB>(p.lv.states, s_off + static_cast<size_t>(r + m * G::kPer) * N, s[m]);
    if (G::owns(lane))
        store_out(p.in.o, p.in.o_bf16, static_cast<size_t>(unit) * p.lv.p + mine, p.in.d ? __fmaf_rn(d, x_own, y) : y);
}

// ------------------------------------------------------------ runs of tokens

constexpr int kGroup = 16;  // tokens staged per pass

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
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
template <int N, bool SB, bool IB>
struct Stage {
    using Elem = typename std::conditional<IB, uint16_t, float>::type;
    Elem b[kGroup][N], c[kGroup][N];
    Elem x[kGroup][Geo<N, SB>::kTile];
    StepScalars sc[kGroup];
};

// A run of tokens on the rows of one CTA, held in registers throughout.  The inputs of 16 tokens
// are staged at a time, the next 16 arriving meanwhile.  With step_snap_ids the state after
// every token is streamed to its snapshot.  A multi-token decode on a bf16-state pool (STEPS) rounds the
// state after every token, as single steps do; a prefill rounds only what it stores at the end.
template <int N, bool SB, bool IB, bool STEPS>
__global__ void __launch_bounds__(kThreads) ssm_run_kernel(const SsmRunArgs p, int tiles) {
    using G = Geo<N, SB>;
    using Elem = typename Stage<N, SB, IB>::Elem;
    __shared__ __align__(16) Stage<N, SB, IB> st[2];
    pdl_prologue();
    const int unit = blockIdx.x / tiles, tile = blockIdx.x - unit * tiles;
    const int bi = unit / p.lv.heads, h = unit - bi * p.lv.heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = warp * G::kWarpRows + lane / G::kLanes;  // this lane's first row in the tile
    const int c0 = (lane & (G::kLanes - 1)) * G::kCols;
    const int slot = __ldg(p.slot_ids + bi);
    if (slot < 0 || slot >= p.lv.n_slots) {
        if (threadIdx.x == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SLOT);
        return;
    }
    long long t0 = static_cast<long long>(bi) * p.n_tok;
    int len = p.n_tok;
    if (!STEPS && p.all_or_none) {
        bool bad = false;
        for (int s = threadIdx.x; s < p.n; s += kThreads) bad |= no_range(p, s);
        if (__syncthreads_or(bad)) {
            if (threadIdx.x == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SEQLENS);
            return;
        }
    }
    if (p.cu_seqlens) {
        const int a = __ldg(p.cu_seqlens + bi), b = __ldg(p.cu_seqlens + bi + 1);
        if (a < 0 || b < a || b > p.total_tokens || b - a > p.max_seqlen) {
            if (threadIdx.x == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SEQLENS);
            return;
        }
        t0 = a;
        len = b - a;
        if (len == 0) return;
    }
    const size_t head_off = p.lv.layer_off + (static_cast<size_t>(h) * p.lv.p + static_cast<size_t>(tile) * G::kTile) * N + c0;
    const size_t s_off = static_cast<size_t>(slot) * p.lv.slot_stride + head_off;
    float s[G::kRows][G::kCols];
#pragma unroll
    for (int m = 0; m < G::kRows; ++m) load_row<G, SB>(p.lv.states, s_off + static_cast<size_t>(r + m * G::kPer) * N, s[m]);
    const float d = p.in.d ? __ldg(p.in.d + h) : 0.f;
    const int g = h / (p.lv.heads / p.lv.groups);
    float raw = 0.f;  // a group's dt, a token a thread
    auto stage = [&](int buf, int first) {
        Stage<N, SB, IB> &to = st[buf];
        const int n = min(kGroup, len - first);
        constexpr int kVec = 16 / static_cast<int>(sizeof(Elem));  // elements per 16 bytes
        constexpr int kState = N / kVec, kTile = G::kTile / kVec, kPerToken = 2 * kState + kTile;
        for (int e = threadIdx.x; e < n * kPerToken; e += kThreads) {
            const int t = e / kPerToken, at = e - t * kPerToken;
            const long long row = t0 + first + t;
            if (at < kState)
                cp_async16(&to.b[t][at * kVec], static_cast<const Elem *>(p.in.b) + row * p.in.b_stride +
                                                    static_cast<long long>(g) * N + at * kVec);
            else if (at < 2 * kState)
                cp_async16(&to.c[t][(at - kState) * kVec], static_cast<const Elem *>(p.in.c) + row * p.in.c_stride +
                                                               static_cast<long long>(g) * N + (at - kState) * kVec);
            else
                cp_async16(&to.x[t][(at - 2 * kState) * kVec],
                           static_cast<const Elem *>(p.in.x) + row * p.in.x_stride + static_cast<long long>(h) * p.lv.p +
                               tile * G::kTile + (at - 2 * kState) * kVec);
        }
        if (threadIdx.x < n) raw = load_dt(p.in, t0 + first + threadIdx.x, h);
    };
    auto scalars = [&](int buf) {
        if (threadIdx.x < kGroup) st[buf].sc[threadIdx.x] = step_scalars(p.in, h, raw);
    };
    stage(0, 0);
    cp_async_commit();
    scalars(0);
    const int own = warp * G::kWarpRows + lane / G::kLanes + G::own_row(lane) * G::kPer;
#pragma unroll 1
    for (int first = 0, buf = 0; first < len; first += kGroup, buf ^= 1) {
        const int n = min(kGroup, len - first);
        const bool more = first + kGroup < len;
        if (more) stage(buf ^ 1, first + kGroup);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        const Stage<N, SB, IB> &at = st[buf];
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
            float b[G::kCols], c[G::kCols], x[G::kRows];
            load_in<G, IB>(at.b[t], c0, b);
            load_in<G, IB>(at.c[t], c0, c);
#pragma unroll
            for (int m = 0; m < G::kRows; ++m) x[m] = widen(at.x[t][r + m * G::kPer]);
            const float y = token_step<G, SB>(s, b, c, x, at.sc[t], lane);
            const long long row = t0 + first + t;
            if (G::owns(lane))
                store_out(p.in.o, p.in.o_bf16, (static_cast<size_t>(row) * p.lv.heads + h) * p.lv.p + tile * G::kTile + own,
                          p.in.d ? __fmaf_rn(d, widen(at.x[t][own]), y) : y);
            if constexpr (STEPS && SB) {
#pragma unroll
                for (int m = 0; m < G::kRows; ++m)
#pragma unroll
                    for (int e = 0; e < G::kCols; ++e) s[m][e] = round_bf16(s[m][e]);
            }
            if (STEPS && p.step_snap_ids) {
                const int id = __ldg(p.step_snap_ids + row);
                if (id < 0 || id >= p.lv.n_snaps) {
                    if (threadIdx.x == 0) flag_status(p.lv.status, WKV7_DEV_BAD_SLOT);
                    continue;
                }
                const size_t d_off = static_cast<size_t>(id) * p.lv.slot_stride + head_off;
#pragma unroll
                for (int m = 0; m < G::kRows; ++m)
                    store_row<G, SB>(p.lv.snaps, d_off + static_cast<size_t>(r + m * G::kPer) * N, s[m]);
            }
        }
        if (more) scalars(buf ^ 1);
        __syncthreads();  // this buffer is refilled by the next pass
    }
#pragma unroll
    for (int m = 0; m < G::kRows; ++m) store_row<G, SB>(p.lv.states, s_off + static_cast<size_t>(r + m * G::kPer) * N, s[m]);
}

template <int N, bool SB, bool IB>
cudaError_t step_as(const SsmRunArgs &a, cudaStream_t s, bool single) {
    const int tiles = a.lv.p / Geo<N, SB>::kTile;
    const long long ctas = static_cast<long long>(a.n) * a.lv.heads * tiles;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto kernel = single ? ssm_decode_kernel<N, SB, IB>
                         : a.cu_seqlens ? ssm_run_kernel<N, SB, IB, false> : ssm_run_kernel<N, SB, IB, true>;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, s, a, tiles);
}

cudaError_t dispatch(const SsmRunArgs &a, cudaStream_t s, int *launches, bool single) {
    cudaError_t (*const as[8])(const SsmRunArgs &, cudaStream_t, bool) = {
        step_as<64, false, false>,  step_as<64, false, true>,  step_as<64, true, false>,  step_as<64, true, true>,
        step_as<128, false, false>, step_as<128, false, true>, step_as<128, true, false>, step_as<128, true, true>};
    const cudaError_t e = as[(a.lv.ds == 128 ? 4 : 0) | (a.lv.state_bf16 ? 2 : 0) | (a.in.bf16 ? 1 : 0)](a, s, single);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssm_decode(const SsmRunArgs &a, cudaStream_t s, int *launches) { return dispatch(a, s, launches, true); }
cudaError_t launch_ssm_run(const SsmRunArgs &a, cudaStream_t s, int *launches) { return dispatch(a, s, launches, false); }

}  // namespace wkv7
