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

constexpr int kThreads = 256;  // four CTAs an SM (64 registers)
constexpr int kMaxCluster = 8;  // portable

struct Best {
    float score = -1.f;  // of no entry
    int at = 0;
    // Larger is better, the lower index among equals; 0 for no entry.
    __device__ __forceinline__ unsigned long long key() const {
        return score < 0.f ? 0ull
                           : (static_cast<unsigned long long>(__float_as_uint(score) + 1u) << 32) |
                                 (0xffffffffu - static_cast<uint32_t>(at));
    }
};

// The division is taken only where it can matter: r <= f * noise, rounded down, proves
// that r / noise rounds to at most f.  f is the thread's own best (its entries arrive in
// rising order, so the earlier of two equal ones stays) or, if larger, the number before
// the best of the whole CTA so far (whose index may be the higher one, so an equal score
// still counts).  After the first entries hardly any pass: an entry costs a subtraction, a
// product and a comparison (with the division inlined and the thread's own best alone it was
// 58 instructions, and 60 and 21 us instead of the launcher's 49 and 8 in the same measurement).
struct Search {
    Best best;
    uint32_t *bar;  // shared: score bits of the CTA's best so far, 0 for none

    __device__ __forceinline__ float bound() const {
        const uint32_t b = *reinterpret_cast<volatile uint32_t *>(bar);
        return fmaxf(best.score, b ? __uint_as_float(b - 1u) : -1.f);
    }
    // U entries, the i-th at index x + i * step; every lane of the warp comes here.
    template <int U>
    __device__ __forceinline__ void take(const float (&r)[U], const float (&noise)[U], int x, int step) {
        float f = bound();
        bool pass = false;
#pragma unroll
        for (int i = 0; i < U; ++i) pass |= r[i] > __fmul_rd(f, noise[i]);  // (NaN: no)
        if (!__any_sync(0xffffffffu, pass)) return;
        if (pass) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (r[i] > 0.f && r[i] > __fmul_rd(f, noise[i])) {
                    const float score = __fdiv_rn(r[i], noise[i]);
                    if (score > best.score) {
                        best.score = score;
                        best.at = x + i * step;
                        f = fmaxf(f, score);
                    }
                }
            }
        }
        const uint32_t m = __reduce_max_sync(0xffffffffu, best.score > 0.f ? __float_as_uint(best.score) : 0u);
        if ((threadIdx.x & 31) == 0) atomicMax(bar, m);
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
// A CTA may reach into another one's shared memory only once that one has begun to run, which being
// launched as one cluster does not give: every thread says at the kernel's start that it has begun
// and waits for the others' word before the first remote store (and before an early return,
// so that the pairs match).
__device__ __forceinline__ void cluster_begun() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait_begun() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote_u64(void *local, uint32_t rank, unsigned long long v) {
    const uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local));
    uint32_t b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(b), "l"(v) : "memory");
}

// What is subtracted from the target's row: nothing, the draft's row, or the whole of
// one entry.
enum { kNothing, kRow, kOne };

// This thread's best entry of [x0, x1), x0 a multiple of 8.  All threads come to it.
template <bool PB, int MINUS>
__device__ __forceinline__ Best scan(const void *p, const void *q, const float *noise, int without, int x0, int x1,
                                     uint32_t *bar) {
    Search search{Best{}, bar};
    const bool aligned = ((reinterpret_cast<uintptr_t>(p) | (MINUS == kRow ? reinterpret_cast<uintptr_t>(q) : 0) |
                           reinterpret_cast<uintptr_t>(noise)) & 15) == 0;
    auto rest = [&](float pv, float qv, int x) {
        return MINUS == kRow ? pv - qv : (MINUS == kOne && x == without) ? 0.f : pv;
    };
    int y0 = x0;
    if (aligned) {  // 8 entries a thread: 16 bytes of bf16, twice that of float32
        for (; y0 + kThreads * 8 <= x1; y0 += kThreads * 8) {
            const int y = y0 + static_cast<int>(threadIdx.x) * 8;
            float pv[8], qv[8], nv[8];
            load8<PB>(p, y, pv);
            if (MINUS == kRow) load8<PB>(q, y, qv);
            load8<false>(noise, y, nv);
#pragma unroll
            for (int i = 0; i < 8; ++i) pv[i] = rest(pv[i], MINUS == kRow ? qv[i] : 0.f, y + i);
            search.take(pv, nv, y, 1);
        }
    } else {
        for (; y0 + kThreads * 8 <= x1; y0 += kThreads * 8) {
            const int y = y0 + static_cast<int>(threadIdx.x);
            float pv[8], qv[8], nv[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                pv[i] = load1<PB>(p, y + i * kThreads);
                if (MINUS == kRow) qv[i] = load1<PB>(q, y + i * kThreads);
                nv[i] = __ldg(noise + y + i * kThreads);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) pv[i] = rest(pv[i], MINUS == kRow ? qv[i] : 0.f, y + i * kThreads);
            search.take(pv, nv, y, kThreads);
        }
    }
    if (y0 < x1) {  // what is left, fewer than 8 entries a thread
        float pv[8], nv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int x = y0 + i * kThreads + static_cast<int>(threadIdx.x);
            const bool in = x < x1;
            pv[i] = in ? rest(load1<PB>(p, x), MINUS == kRow ? load1<PB>(q, x) : 0.f, x) : 0.f;
            nv[i] = in ? __ldg(noise + x) : 1.f;
        }
        search.take(pv, nv, y0 + static_cast<int>(threadIdx.x), kThreads);
    }
    return search.best;
}

template <bool PB>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyArgs a) {
    __shared__ unsigned long long warp_best[kThreads / 32];
    __shared__ unsigned long long from[2][kMaxCluster];  // by pass
    __shared__ int sh_m, sh_bad;
    __shared__ uint32_t sh_bar[2];  // by pass
    cluster_begun();
    if (threadIdx.x < 2) sh_bar[threadIdx.x] = 0;
    pdl_wait();  // and no early start for the next kernel: it may read the ids chosen here before its own wait
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
        for (int j0 = 0; j0 < K; j0 += 32) {
            const int j = j0 + lane;
            bool ok = false, out = false;
            if (j < K) {  // read beside the row's count, not after it
                const int id = __ldg(d.draft_ids + static_cast<long long>(row) * K + j);
                const float u = __ldg(d.uniforms + static_cast<long long>(row) * K + j);
                out = id < 0 || id >= d.vocab;
                if (!out) {
                    const float pd = load1<PB>(d.p, p_row0 + j * d.p_row_stride + id);
                    const float qd = d.q ? load1<PB>(d.q, q_row0 + j * d.q_row_stride + id) : 1.f;
                    ok = __fmul_rn(u, qd) < pd && j < drafted;
                }
                out = out && j < drafted;
            }
            if (!bad && __any_sync(0xffffffffu, out)) bad = WKV7_DEV_BAD_TOKEN;
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
    cluster_wait_begun();
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
        uint32_t *bar = &sh_bar[pass];
        if (pass == 0 && q)
            best = scan<PB, kRow>(p, q, noise, -1, x0, x1, bar).key();
        else if (pass == 0 && without >= 0)
            best = scan<PB, kOne>(p, nullptr, noise, without, x0, x1, bar).key();
        else
            best = scan<PB, kNothing>(p, nullptr, noise, -1, x0, x1, bar).key();
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
    // CTAs per row: two or more for each SM in all, and more than 2,048 entries each (a row is split
    // while its parts have over 4,096).  In a graph, 1 row of 65,536 / 256 of 130,001 / 64 of 65,529
    // (bf16, misaligned) take 5.7 / 48.0 / 7.0 us, the second 0.29 GB at 6.0 TB/s.  When the shape was chosen it was 5.5 / 49.1 / 8.3; with four
    // times as many CTAs 5.5 / 58.1 / 8.1 (each row's start is three dependent reads), with 512
    // threads a CTA 5.4 / 52.2 / 12.5, 1,024 5.9 / 62.8 / 25.8.
    int size = 1;
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
