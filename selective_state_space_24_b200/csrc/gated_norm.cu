// gated_norm.cu -- RMS norm of groups of channels with a SiLU gate, and its
// gradients.  Per group of g channels, s = silu(z):
//     gate first:  u = x s,  n = u r,  out = n w
//     norm first:  u = x,    n = u r,  out = n w s        r = (mean u^2 + eps)^-1/2
// Backward, dn = dout w (gate first) or dout w s (norm first):
//     du = r (dn - n mean(dn n)),  dw = sum over rows of dn n / w
//     gate first:  dx = du s, dz = du x s';   norm first:  dx = du, dz = dout n w s'
// with s' = sigmoid(z) (1 + z (1 - sigmoid(z))).  Both sums of the backward
// (u^2 and dn u, as mean(dn n) = r mean(dn u)) are taken in one reduction.
//
// Bound by HBM: every operand passes once, a row stays in registers between
// its loads and its stores.  A thread keeps the same columns for every row it
// meets (NormPlan), so the weights are read once per thread and dw gathers in
// registers; each block then writes one partial row of dw, summed by a second
// small kernel in a fixed order (no atomics: the same bits every time).
#include "norm_common.cuh"

namespace ssm {
namespace {

NormPlan gated_plan(int64_t rows, int dim, int group)
{
    const int G = dim / group;
    NormPlan p = norm_threads(group);
    const int64_t need = (rows + p.rows_at_once - 1) / p.rows_at_once;
    const int64_t most = ((int64_t)148 * (2048 / p.threads) + G - 1) / G;
    p.parts = (int)(need < most ? need : most);
    return p;
}

template <typename T, bool BWD>
__global__ void __launch_bounds__(512) gated_norm_kernel(const GatedArgs a, int tpr, int rpb, int parts)
{
    constexpr int E = Vec<T>::N, NV = kNormElems / E;
    __shared__ RedSmem red;
    extern __shared__ float cols[];   // (group), backward only
    const int lane_r = threadIdx.x % tpr, sub = threadIdx.x / tpr;
    const int nv = a.group / E, G = a.dim / a.group;
    const int part = blockIdx.x / G;
    const int col = (int)(blockIdx.x % G) * a.group;
    const T *x = static_cast<const T *>(a.x), *z = static_cast<const T *>(a.z);
    const T *dout = static_cast<const T *>(a.dout);
    const float inv = 1.f / (float)a.group;
    int turn = 0;

    float w[NV][E], dw[NV][E];
    bool in[NV];
#pragma unroll
    for (int v = 0; v < NV; v++) {
        in[v] = lane_r + v * tpr < nv;
#pragma unroll
        for (int e = 0; e < E; e++)
            w[v][e] = dw[v][e] = 0.f;
        if (in[v])
            load_f32<E>(a.weight + col + (lane_r + v * tpr) * E, w[v]);
    }
    // every thread of the block takes the same number of turns (barriers)
    for (int64_t r0 = (int64_t)part * rpb; r0 < a.rows; r0 += (int64_t)parts * rpb) {
        const bool live = r0 + sub < a.rows;
        const int64_t base = (r0 + sub) * a.dim + col;
        float xv[NV][E], zv[NV][E], dv[NV][E];
#pragma unroll
        for (int v = 0; v < NV; v++) {
            const int64_t at = base + (lane_r + v * tpr) * E;
#pragma unroll
            for (int e = 0; e < E; e++)
                xv[v][e] = zv[v][e] = dv[v][e] = 0.f;
            if (live && in[v]) {
                Vec<T>::load(x + at, xv[v]);
                if (z)
                    Vec<T>::load(z + at, zv[v]);
                if (BWD)
                    Vec<T>::load(dout + at, dv[v]);
            }
        }
        float sg[NV][E];   // sigmoid(z)
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int e = 0; e < E; e++) {
                sg[v][e] = z ? sigmoid_f(zv[v][e]) : 1.f;
                const float s = z ? zv[v][e] * sg[v][e] : 1.f;
                const float u = a.norm_first ? xv[v][e] : xv[v][e] * s;
                sum[0] = fmaf(u, u, sum[0]);
                if (BWD) {
                    const float dn = a.norm_first ? dv[v][e] * s * w[v][e] : dv[v][e] * w[v][e];
                    sum[1] = fmaf(dn, u, sum[1]);
                }
            }
        if (BWD) {
            row_sum<2>(sum, tpr, red, turn);
        } else {
            float one[1] = {sum[0]};
            row_sum<1>(one, tpr, red, turn);
            sum[0] = one[0];
        }
        const float r = rsqrtf(sum[0] * inv + a.eps);
        const float m = sum[1] * inv * r;   // mean(dn n)
#pragma unroll
        for (int v = 0; v < NV; v++) {
            const int64_t at = base + (lane_r + v * tpr) * E;
            float o[E], oz[E];
#pragma unroll
            for (int e = 0; e < E; e++) {
                const float zz = zv[v][e], s = z ? zz * sg[v][e] : 1.f;
                const float u = a.norm_first ? xv[v][e] : xv[v][e] * s, n = u * r;
                if (!BWD) {
                    o[e] = a.norm_first ? n * w[v][e] * s : n * w[v][e];
                } else {
                    const float ds = sg[v][e] * fmaf(zz, 1.f - sg[v][e], 1.f);
                    const float dy = a.norm_first ? dv[v][e] * s : dv[v][e];
                    dw[v][e] = fmaf(dy, n, dw[v][e]);
                    const float du = r * fmaf(-n, m, dy * w[v][e]);
                    o[e] = a.norm_first ? du : du * s;
                    oz[e] = (a.norm_first ? dv[v][e] * n * w[v][e] : du * xv[v][e]) * ds;
                }
            }
            if (live && in[v]) {
                Vec<T>::store(static_cast<T *>(BWD ? a.dx : a.out) + at, o);
                if (BWD && z)
                    Vec<T>::store(static_cast<T *>(a.dz) + at, oz);
            }
        }
    }
    if (BWD) {
        // one partial row of dw per block, its rows added in the order of
        // their threads
        for (int s = 0; s < rpb; s++) {
            if (s == sub)
#pragma unroll
                for (int v = 0; v < NV; v++)
                    if (in[v])
#pragma unroll
                        for (int e = 0; e < E; e++) {
                            const int c = (lane_r + v * tpr) * E + e;
                            cols[c] = s == 0 ? dw[v][e] : cols[c] + dw[v][e];
                        }
            __syncthreads();
        }
        float *out = a.parts + (size_t)part * a.dim + col;
        for (int c = threadIdx.x; c < a.group; c += blockDim.x)
            out[c] = cols[c];
    }
}

template <typename T, bool BWD> cudaError_t launch_typed(const GatedArgs &a, cudaStream_t st)
{
    const NormPlan p = gated_plan(a.rows, a.dim, a.group);
    const unsigned blocks = (unsigned)p.parts * (unsigned)(a.dim / a.group);
    gated_norm_kernel<T, BWD><<<blocks, p.threads, BWD ? a.group * sizeof(float) : 0, st>>>(a, p.tpr, p.rows_at_once, p.parts);
    return cudaGetLastError();
}

// 32 columns x 8 strands of partial rows; the strands are joined in order
__global__ void __launch_bounds__(256) part_sum_kernel(const float *parts, int nparts, int dim, float *out)
{
    __shared__ float s[8][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    const float *p = parts + (size_t)blockIdx.y * nparts * dim;
    float v = 0.f;
    if (c < dim)
        for (int k = threadIdx.y; k < nparts; k += 8)
            v += p[(size_t)k * dim + c];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && c < dim) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; k++)
            t += s[k][threadIdx.x];
        out[(size_t)blockIdx.y * dim + c] = t;
    }
}

}  // namespace

cudaError_t launch_part_sum(const float *parts, int64_t sets, int nparts, int dim, float *out, cudaStream_t st)
{
    for (int64_t s = 0; s < sets; s += 65535) {
        const unsigned n = (unsigned)(sets - s < 65535 ? sets - s : 65535);
        part_sum_kernel<<<dim3((dim + 31) / 32, n), dim3(32, 8), 0, st>>>(parts + (size_t)s * nparts * dim, nparts, dim,
                                                                         out + (size_t)s * dim);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

size_t gated_bwd_workspace(int64_t rows, int dim, int group)
{
    return (size_t)gated_plan(rows, dim, group).parts * dim * sizeof(float);
}

cudaError_t launch_gated_fwd(const GatedArgs &a, cudaStream_t st)
{
    return a.dtype == 0 ? launch_typed<float, false>(a, st) : launch_typed<__nv_bfloat16, false>(a, st);
}

cudaError_t launch_gated_bwd(const GatedArgs &a, cudaStream_t st)
{
    const cudaError_t e =
        a.dtype == 0 ? launch_typed<float, true>(a, st) : launch_typed<__nv_bfloat16, true>(a, st);
    if (e != cudaSuccess)
        return e;
    return launch_part_sum(a.parts, 1, gated_plan(a.rows, a.dim, a.group).parts, a.dim, a.dweight, st);
}

}  // namespace ssm
