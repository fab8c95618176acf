// Gates: x sigmoid(x) and sigmoid(x) from the approximate 2^x and reciprocal (a few units in the
// last place of float32; the exact functions made the gated norm of long inputs instruction-bound).
#pragma once

#include <cuda_runtime.h>

namespace wkv7 {

__device__ __forceinline__ float sigmoid(float x) {
    float e, y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + e));
    return y;
}
// (-inf gives NaN, as the product does; below about -88 the reciprocal of infinity is 0.)
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }

}  // namespace wkv7
