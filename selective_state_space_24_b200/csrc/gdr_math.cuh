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
// below 2^-150 is zero, so the logarithm stops there: an infinite one would
// leave NaN in the sums.  NaN stays NaN.
__device__ __forceinline__ float gdr_log_decay(float dt, float A_log2e)
{
    const float g = dt * A_log2e;
    return g < -150.f ? -150.f : g;
}
// The sum of two numbers hi + lo (x, y): hi's rounding error, found by adding
// backwards, goes to lo.
__device__ __forceinline__ float2 pair_add(float2 a, float2 b)
{
    const float s = __fadd_rn(a.x, b.x), v = __fsub_rn(s, a.x);
    const float e = __fadd_rn(__fsub_rn(a.x, __fsub_rn(s, v)), __fsub_rn(b.x, v));
    return make_float2(s, __fadd_rn(__fadd_rn(a.y, b.y), e));
}
// The sums of a chunk's 64 log decays up to and with steps 2 l and 2 l + 1, for
// lane l, which has their values; as pairs, because every decay between two
// steps is a difference of two sums: with float32 sums it would lose what
// their magnitude costs (sums in the thousands, where sequences of a few steps
// are packed: 4e-4 of a decay; ordinary gates of 2 bits a step 3e-5; pairs
// 1e-6, the rounding of the difference itself).
__device__ __forceinline__ void gdr_log_sums(const float (&g)[2], float2 (&cs)[2])
{
    const int lane = threadIdx.x & 31;
    const float2 first = make_float2(g[0], 0.f);
    float2 incl = pair_add(first, make_float2(g[1], 0.f));
    auto from_below = [&](int o) {
        return make_float2(__shfl_up_sync(0xffffffffu, incl.x, o), __shfl_up_sync(0xffffffffu, incl.y, o));
    };
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {   // (small code: see gdr_chunk.cu)
        const float2 u = from_below(o);
        if (lane >= o)
            incl = pair_add(u, incl);
    }
    const float2 before = from_below(1);
    cs[0] = lane > 0 ? pair_add(before, first) : first;
    cs[1] = incl;
#pragma unroll
    for (int i = 0; i < 2; i++) {   // lo at most half a step of hi
        const float hi = __fadd_rn(cs[i].x, cs[i].y);
        cs[i] = make_float2(hi, __fadd_rn(__fsub_rn(cs[i].x, hi), cs[i].y));
    }
}
// 2^(n lo), n at most 2: a lo is at most 2^-11 (half a step of 64 * 150), so
// what its square would add stays below 2^-22 there, and far below elsewhere.
__device__ __forceinline__ float gdr_rest(float n, float lo) { return fmaf(n * 0.69314718f, lo, 1.f); }
// The decay between two such sums, later and earlier.
__device__ __forceinline__ float gdr_between(float hi, float lo, float hi0, float lo0)
{
    return ex2_mufu((hi - hi0) + (lo - lo0));
}

}  // namespace ssm
