// What a token contributes to a head of the selective scan besides x, B and C.
#pragma once

#include "device_common.cuh"
#include "ssm_internal.h"

namespace wkv7 {

struct StepScalars {
    float dt;  // the step, after bias and softplus
    float a;   // exp(dt A)
};

__device__ __forceinline__ float load_dt(const SsmTokens &in, long long row, int h) {
    const size_t at = static_cast<size_t>(row * in.dt_stride + h);
    return in.dt_bf16 ? load1<true>(in.dt, at) : load1<false>(in.dt, at);
}

// log(1 + e^x); above 20 e^-x is below float32's resolution of x.
__device__ __forceinline__ float softplus(float x) { return x > 20.f ? x : log1pf(expf(x)); }

__device__ __forceinline__ float step_size(const SsmTokens &in, int h, float raw) {
    const float x = in.dt_bias ? __fadd_rn(raw, __ldg(in.dt_bias + h)) : raw;
    return in.softplus ? softplus(x) : x;
}
__device__ __forceinline__ StepScalars step_scalars(const SsmTokens &in, int h, float raw) {
    StepScalars t;
    t.dt = step_size(in, h, raw);
    t.a = expf(__fmul_rn(t.dt, __ldg(in.a + h)));
    return t;
}

// Whether sequence s of a call is no range of its tokens.
__device__ __forceinline__ bool no_range(const SsmRunArgs &p, int s) {
    const int a = __ldg(p.cu_seqlens + s), b = __ldg(p.cu_seqlens + s + 1);
    return a < 0 || b < a || b > p.total_tokens;
}

}  // namespace wkv7
