// Verification of drafted tokens against the target's probabilities, from given
// random numbers.
//
// A row's m accepted drafts follow from K scattered probabilities; its next token
// is the argmax over the vocabulary of r_x / noise_x with r = max(p_m - q_m, 0),
// which for exponential noise is a sample of the normalised r (the smallest of
// independent exponentials of rates r_x).  Neither needs a sum over the
// vocabulary, so every value is one correctly rounded operation and the result
// does not depend on how the row is split.
//
// Bound by HBM: one pass over p_m, q_m and the noise, 12 bytes per entry.  A row
// is split over a cluster of CTAs that exchange their best entry through
// distributed shared memory: one launch, no workspace.
#include "device_common.cuh"
#include "wkv7_internal.h"

namespace wkv7 {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxCluster = 8;  // portable

struct Best {
    float score = -1.f;  // of no entry
    int at = 0;
    // The division only where it can matter: r <= score * noise, rounded down,
    // proves that r / noise is no larger.  Entries arrive in rising order, so the
    // earlier of two equal ones stays.
    __device__ __forceinline__ void take(float r, float noise, int x) {
        if (r > 0.f && !(r <= __fmul_rd(score, noise))) {
            const float f = __fdiv_rn(r, noise);
            if (f > score) {
                score = f;
                at = x;
            }
        }
    }
    // Larger is better, the lower index among equals; 0 for no entry.
    __device__ __forceinline__ unsigned long long key() const {
        return score < 0.f ? 0ull
                           : (static_cast<unsigned long long>(__float_as_uint(score) + 1u) << 32) |
                                 (0xffffffffu - static_cast<uint32_t>(at));
    }
};

template <bool PB>
__device__ __forceinline__ const void *entry(const void *p, long long off) {
    return PB ? static_cast<const void *>(static_cast<const uint16_t *>(p) + off)
              : static_cast<const void *>(static_cast<const float *>(p) + off);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote_u64(void *local, uint32_t rank, unsigned long long v) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    uint32_t b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(b), "l"(v) : "memory");
}

// This thread's best entry of [x0, x1): max(p - q, 0) / noise (q may be null; at
// `without`, p counts as 0).
template <bool PB>
__device__ __forceinline__ Best scan(const void *p, const void *q, const float *noise, int without, int x0, int x1) {
    Best best;
    auto residual = [&](float pv, float qv, int x) { return x == without ? 0.f : pv - qv; };
    const bool aligned = ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q) |
                           reinterpret_cast<uintptr_t>(noise)) & 15) == 0;
    constexpr int V = PB ? 8 : 4;  // entries of 16 bytes of p
    int x = x0 + static_cast<int>(threadIdx.x);
    if (aligned) {  // x0 is a multiple of 8
        const int vec_end = x0 + (x1 - x0) / V * V;
#pragma unroll 2
        for (int y = x0 + static_cast<int>(threadIdx.x) * V; y < vec_end; y += kThreads * V) {
            float pv[V], qv[V], nv[V];
            if constexpr (PB) {
                load8<true>(p, y, pv);
                if (q) load8<true>(q, y, qv);
                load8<false>(noise, y, nv);
            } else {
                const float4 a = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + y));
                const float4 c = __ldg(reinterpret_cast<const float4 *>(noise + y));
                pv[0] = a.x; pv[1] = a.y; pv[2] = a.z; pv[3] = a.w;
                nv[0] = c.x; nv[1] = c.y; nv[2] = c.z; nv[3] = c.w;
                if (q) {
                    const float4 b = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(q) + y));
                    qv[0] = b.x; qv[1] = b.y; qv[2] = b.z; qv[3] = b.w;
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) best.take(residual(pv[i], q ? qv[i] : 0.f, y + i), nv[i], y + i);
        }
        x = vec_end + static_cast<int>(threadIdx.x);
    }
#pragma unroll 4
    for (; x < x1; x += kThreads)
        best.take(residual(load1<PB>(p, x), q ? load1<PB>(q, x) : 0.f, x), __ldg(noise + x), x);
    return best;
}

template <bool PB>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a) {
    __shared__ unsigned long long warp_best[kThreads / 32];
    __shared__ unsigned long long from[2][kMaxCluster];  // by pass
    __shared__ int sh_m, sh_bad;
    pdl_prologue();
    const wkv7_draft_batch &d = a.d;
    const int rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
    const int row = blockIdx.x / size;
    const int K = d.n_draft;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int drafted = d.n_draft_rows ? __ldg(d.n_draft_rows + row) : K;
    const long long p_row0 = static_cast<long long>(row) * d.p_batch_stride;
    const long long q_row0 = static_cast<long long>(row) * d.q_batch_stride;
    if (warp == 0) {
        int m = 0, bad = (drafted < 0 || drafted > K) ? WKV7_DEV_BAD_SEQLENS : 0;
        bool open = true;  // no draft refused so far
        for (int j0 = 0; !bad && j0 < drafted; j0 += 32) {
            const int j = j0 + lane;
            bool ok = false, out = false;
            if (j < drafted) {
                const int id = __ldg(d.draft_ids + static_cast<long long>(row) * K + j);
                out = id < 0 || id >= d.vocab;
                if (!out) {
                    const float pd = load1<PB>(d.p, p_row0 + j * d.p_row_stride + id);
                    const float qd = d.q ? load1<PB>(d.q, q_row0 + j * d.q_row_stride + id) : 1.f;
                    ok = __fmul_rn(__ldg(d.uniforms + static_cast<long long>(row) * K + j), qd) < pd;
                }
            }
            if (__any_sync(0xffffffffu, out)) bad = WKV7_DEV_BAD_TOKEN;
            const unsigned yes = __ballot_sync(0xffffffffu, ok);
            const int run = yes == 0xffffffffu ? 32 : __ffs(~yes) - 1;
            if (open) m += run;
            open = open && run == 32;
        }
        if (lane == 0) {
            sh_m = m;
            sh_bad = bad;
        }
    }
    __syncthreads();
    const int m = sh_m, bad = sh_bad;
    int *tokens = d.tokens + static_cast<long long>(row) * (K + 1);
    if (bad) {  // the same in every CTA of the cluster
        if (rank == 0) {
            for (int j = threadIdx.x; j <= K; j += kThreads) tokens[j] = -1;
            if (threadIdx.x == 0) {
                d.accepted[row] = -1;
                if (d.resume_ids) d.resume_ids[row] = -1;
                flag_status(a.status, bad);
            }
        }
        return;
    }
    const bool refused = m < drafted;
    const void *p = entry<PB>(d.p, p_row0 + static_cast<long long>(m) * d.p_row_stride);
    const void *q = refused && d.q ? entry<PB>(d.q, q_row0 + static_cast<long long>(m) * d.q_row_stride) : nullptr;
    const float *noise = d.noise + static_cast<long long>(row) * d.noise_stride;
    const int without = refused && !d.q ? __ldg(d.draft_ids + static_cast<long long>(row) * K + m) : -1;
    const int part = (d.vocab / size + 8) / 8 * 8;  // >= vocab / size, a multiple of 8
    const int x0 = min(d.vocab, rank * part), x1 = min(d.vocab, x0 + part);
    unsigned long long best = 0;
    for (int pass = 0; pass < 2; ++pass) {  // the second one, over p alone, only if the residual is empty
        best = (pass == 0 ? scan<PB>(p, q, noise, without, x0, x1) : scan<PB>(p, nullptr, noise, -1, x0, x1)).key();
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, off);
            best = other > best ? other : best;
        }
        if (lane == 0) warp_best[warp] = best;
        __syncthreads();
        if (warp == 0) {
            best = lane < kThreads / 32 ? warp_best[lane] : 0;
#pragma unroll
            for (int off = kThreads / 64; off >= 1; off >>= 1) {
                const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, off);
                best = other > best ? other : best;
            }
            best = __shfl_sync(0xffffffffu, best, 0);
            if (lane < size) store_remote_u64(&from[pass][rank], lane, best);
        }
        cluster_sync();
        best = 0;
        for (int i = 0; i < size; ++i) best = from[pass][i] > best ? from[pass][i] : best;
        if (best != 0 || !refused) break;  // the same in every thread of the cluster
    }
    if (rank != 0) return;
    const int next = best ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(best)) : -1;
    for (int j = threadIdx.x; j <= K; j += kThreads)
        tokens[j] = j < m ? __ldg(d.draft_ids + static_cast<long long>(row) * K + j) : j == m ? next : -1;
    if (threadIdx.x == 0) {
        d.accepted[row] = m;
        if (d.resume_ids) {
            const int id = __ldg(d.step_snap_ids + static_cast<long long>(row) * (K + 1) + m);
            const bool ok = id >= 0 && id < a.n_snaps;
            d.resume_ids[row] = ok ? id : -1;
            if (!ok) flag_status(a.status, WKV7_DEV_BAD_SLOT);
        }
    }
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t s, int *launches) {
    int size = 1;  // CTAs per row: about four for each SM, and at least 4,096 entries each
    while (size < kMaxCluster && static_cast<long long>(a.d.n) * size < 2 * 152 && a.d.vocab / size > 4096) size *= 2;
    const long long ctas = static_cast<long long>(a.d.n) * size;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(size);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, a.d.prob_dtype == WKV7_BF16 ? verify_kernel<true> : verify_kernel<false>, a);
    ++*launches;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace wkv7
