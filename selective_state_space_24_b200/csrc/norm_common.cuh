// norm_common.cuh -- what the norm kernels share: a thread's part of a row,
// sums over the threads of one row (or group), how many blocks to launch.
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
    static __device__ __forceinline__ void unpack(const uint4 &v, float *f)
    {
        f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *f)
    {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &v, float *f)
    {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
            f[2 * k] = __uint_as_float(u[k] << 16);
            f[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *f)
    {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
            u[k] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

// This thread's elements of one row of R as they lie in memory: NV vectors of
// N elements (N as the call's type has in 16 bytes), held until they are used,
// so that the next row's are on their way during the work on this one.
template <typename R, int NV, int N> struct Raw {
    static constexpr int W = N / Vec<R>::N;   // 16-byte words per vector
    uint4 w[NV][W];
    // vectors lane_r, lane_r + tpr, .. of the row at p; zeros outside it (on[v] false)
    __device__ __forceinline__ void load(const R *p, int lane_r, int tpr, const bool (&on)[NV], bool live)
    {
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int k = 0; k < W; k++)
                w[v][k] = live && on[v]
                              ? reinterpret_cast<const uint4 *>(p + (lane_r + v * tpr) * N)[k]
                              : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(int v, float (&f)[N]) const
    {
#pragma unroll
        for (int k = 0; k < W; k++)
            Vec<R>::unpack(w[v][k], &f[k * Vec<R>::N]);
    }
    __device__ __forceinline__ void get(float (&f)[NV][N]) const
    {
#pragma unroll
        for (int v = 0; v < NV; v++)
            get(v, f[v]);
    }
};
template <typename R, int N> __device__ __forceinline__ void store_row(R *p, const float (&f)[N])
{
#pragma unroll
    for (int k = 0; k < N / Vec<R>::N; k++)
        reinterpret_cast<uint4 *>(p)[k] = Vec<R>::pack(&f[k * Vec<R>::N]);
}

constexpr int kSMs = 148;

// Threads for rows of `len` elements normed together.  Eight elements a
// thread (one or two 16-byte words) leave room for several blocks per SM:
// the norm of 128-channel heads (262144 rows, bf16) took 61 us with sixteen
// and 40 with eight and the next row's loads ahead, for which they leave room.
// Rows above 4096 need sixteen to stay within 512 threads, which in the
// gradients (column sums, and the next row) do not fit 128 registers: those
// variants spill, up to 1.9 KB a thread, and take 1.4 to 3.5 times their bytes'
// time.
inline NormPlan norm_threads(int len)
{
    NormPlan p;
    p.elems = len <= 4096 ? 8 : 16;   // up to 512 threads a row
    p.tpr = 1;
    while (p.tpr * p.elems < len)
        p.tpr *= 2;
    p.threads = p.tpr > 128 ? p.tpr : 128;
    p.rows_at_once = p.threads / p.tpr;
    return p;
}

// Blocks of a kernel that the GPU holds at once: blocks that walk their rows
// with a stride are launched that often, so that all of them end together.
template <class Kern> int64_t resident_blocks(Kern kernel, int threads, size_t smem)
{
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n < 1)
        n = 1;
    return (int64_t)kSMs * n;
}

// Blocks for the rows of one group or set, of which there are `shares`: as many
// as rows, at most `most` for all of them together.
inline int64_t parts_for(int64_t rows, int64_t shares, const NormPlan &p, int64_t most)
{
    const int64_t need = (rows + p.rows_at_once - 1) / p.rows_at_once, share = most / shares;
    return share < 1 ? 1 : need < share ? need : share;
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
constexpr int kRedMax = 3;   // values summed at once
// shared memory of row_sum: two buffers in turn, so that one barrier per sum
// is enough (a buffer is written again only after the next sum's barrier)
struct __align__(16) RedSmem {
    float v[2][kRedMax][32];   // one value per warp
};

// Sums v[0..K) over the `tpr` neighbouring threads of this thread's row (a
// power of two) -- each of them gets the same sums, added in the same order.
// With more than 32 threads per row every thread of the block must call it.
template <int K, int M> __device__ __forceinline__ void row_sum(float (&v)[M], int tpr, RedSmem &sm, int &turn)
{
    static_assert(K <= kRedMax && K <= M, "the first K of M values");
    const int in_warp = tpr < 32 ? tpr : 32;
    for (int o = in_warp >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; k++)
            v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (tpr > 32) {   // 2 to 16 warps a row: every thread adds their values itself
        const int nw = tpr >> 5, w0 = (threadIdx.x / tpr) * nw;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < K; k++)
                sm.v[turn][k][threadIdx.x >> 5] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; k++) {
            const float2 a = *reinterpret_cast<const float2 *>(&sm.v[turn][k][w0]);
            v[k] = a.x + a.y;
            for (int i = 2; i < nw; i += 2) {
                const float2 b = *reinterpret_cast<const float2 *>(&sm.v[turn][k][w0 + i]);
                v[k] += b.x + b.y;
            }
        }
        turn ^= 1;
    }
}

// The mean from a sum over n values: the rounded product's remainder, exact in
// one fma, is divided too.  So a row of one value c has the mean c wherever n c
// is a float32.
__device__ __forceinline__ float mean_of(float sum, float n, float inv)
{
    const float q = sum * inv;
    return fmaf(fmaf(-n, q, sum), inv, q);
}

}  // namespace ssm
