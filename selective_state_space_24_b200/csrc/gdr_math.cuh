// gdr_math.cuh -- the scalars of the gated delta rule, shared by its kernels
// so that all of them round alike.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdr.h"
#include "s6_math.cuh"

namespace ssm {

constexpr float kL2Eps = 1e-6f;   // under the root of the 2-norms of q and k

__device__ __forceinline__ float gdr_ld(const float *p, size_t i) { return __ldg(p + i); }
__device__ __forceinline__ float gdr_ld(const __nv_bfloat16 *p, size_t i) { return __bfloat162float(__ldg(p + i)); }
__device__ __forceinline__ void gdr_st(float *p, size_t i, float v) { p[i] = v; }
__device__ __forceinline__ void gdr_st(__nv_bfloat16 *p, size_t i, float v) { p[i] = __float2bfloat16_rn(v); }

__device__ __forceinline__ float gdr_dt(float raw, float bias, int softplus)
{
    const float v = raw + bias;
    return softplus ? softplus_f(v) : v;
}
// One step's log2 decay as the chunked kernels add it up.  A float32 decay
// below 2^-150 is zero, so the logarithm stops there: further out it would
// cost the sums, from which later steps' decays are differences, their low
// bits (one step of -1e5 leaves them 2^-8), and an infinite one would leave
// NaN.  NaN stays NaN.
__device__ __forceinline__ float gdr_log_decay(float dt, float A_log2e)
{
    const float g = dt * A_log2e;
    return g < -150.f ? -150.f : g;
}
// sigmoid(v), also dt's derivative through the softplus
__device__ __forceinline__ float gdr_sigmoid(float v) { return rcp_mufu(1.f + ex2_mufu(-v * kLog2e)); }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace ssm
