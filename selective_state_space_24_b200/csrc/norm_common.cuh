// norm_common.cuh -- what the norm kernels share: vectors of 16 bytes held
// as float32, sums over the threads of one row (or group), and the sum of
// per-CTA partial column sums.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "norm.h"
#include "s6_math.cuh"

namespace ssm {

template <typename T> struct Vec;   // 16 bytes of T
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const float *p, float (&f)[4])
    {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&f)[4])
    {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float (&f)[8])
    {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
            f[2 * k] = __uint_as_float(u[k] << 16);
            f[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&f)[8])
    {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
            u[k] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};

constexpr int kNormElems = 16;      // elements of a row that one thread holds
constexpr int kNormMaxLen = 8192;   // elements normed together: 512 threads of 16

// Threads for rows of `len` elements normed together.
inline NormPlan norm_threads(int len)
{
    NormPlan p;
    p.tpr = 1;
    while (p.tpr * kNormElems < len)
        p.tpr *= 2;
    p.threads = p.tpr > 128 ? p.tpr : 128;
    p.rows_at_once = p.threads / p.tpr;
    p.parts = 1;
    return p;
}

// N consecutive float32 (weights next to a vector of N elements)
template <int N> __device__ __forceinline__ void load_f32(const float *p, float (&f)[N])
{
#pragma unroll
    for (int k = 0; k < N; k += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p + k));
        f[k] = v.x, f[k + 1] = v.y, f[k + 2] = v.z, f[k + 3] = v.w;
    }
}
template <int N> __device__ __forceinline__ void store_f32(float *p, const float (&f)[N])
{
#pragma unroll
    for (int k = 0; k < N; k += 4)
        *reinterpret_cast<float4 *>(p + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
}

// N consecutive elements of the residual stream (float32 or bf16) next to a
// vector of N elements of the call's type
template <typename R, int N> __device__ __forceinline__ void load_row(const R *p, float (&f)[N])
{
#pragma unroll
    for (int k = 0; k < N; k += Vec<R>::N) {
        float t[Vec<R>::N];
        Vec<R>::load(p + k, t);
#pragma unroll
        for (int i = 0; i < Vec<R>::N; i++)
            f[k + i] = t[i];
    }
}
template <typename R, int N> __device__ __forceinline__ void store_row(R *p, const float (&f)[N])
{
#pragma unroll
    for (int k = 0; k < N; k += Vec<R>::N) {
        float t[Vec<R>::N];
#pragma unroll
        for (int i = 0; i < Vec<R>::N; i++)
            t[i] = f[k + i];
        Vec<R>::store(p + k, t);
    }
}

constexpr int kRedMax = 2;   // values summed at once
// shared memory of row_sum: two buffers in turn, so that one barrier per sum
// is enough (a buffer is written again only after the next sum's barrier)
struct RedSmem {
    float v[2][32][kRedMax];
};

// Sums v[0..K) over the `tpr` neighbouring threads of this thread's row (a
// power of two) -- each of them gets the same sums, added in the same order.
// With more than 32 threads per row every thread of the block must call it.
template <int K> __device__ __forceinline__ void row_sum(float (&v)[K], int tpr, RedSmem &sm, int &turn)
{
    static_assert(K <= kRedMax, "");
    const int in_warp = tpr < 32 ? tpr : 32;
    for (int o = in_warp >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; k++)
            v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (tpr > 32) {
        const int nw = tpr >> 5, lane = threadIdx.x & 31, w0 = (threadIdx.x / tpr) * nw;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < K; k++)
                sm.v[turn][threadIdx.x >> 5][k] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; k++)
            v[k] = lane < nw ? sm.v[turn][w0 + lane][k] : 0.f;
        for (int o = nw >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < K; k++)
                v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
#pragma unroll
        for (int k = 0; k < K; k++)
            v[k] = __shfl_sync(0xffffffffu, v[k], 0);
        turn ^= 1;
    }
}

// z sigmoid(z), and with it the sigmoid
__device__ __forceinline__ float sigmoid_f(float z) { return rcp_mufu(1.f + ex2_mufu(-z * kLog2e)); }

}  // namespace ssm
