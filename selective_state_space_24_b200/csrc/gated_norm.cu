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
//
// Measured on B200, bf16: forward, 262144 rows of 128 with a gate 38.5 us
// (5.2 TB/s, 0.80 of a copy; what is missing are the rows' start and the
// sum's round trip per row).  Backward, 16384 rows of 2048: 80 us (4.2 TB/s,
// 0.64): a row's five operands are unpacked, gated and packed at about 14
// instructions an element, and the row's sum joins eight warps at a barrier,
// which four blocks of 256 threads per SM cover in part.  float32: 61 us forward
// (1.0 of a copy), 110 backward (0.93).  Rows above 4096 spill (norm_threads):
// backward, 4096 rows of 8192, bf16 125 us (0.41), float32 185 (0.55).
#include "norm_common.cuh"

namespace ssm {
namespace {

// GATE: 0 none, 1 before the norm, 2 after it (a variant each: tests of it for
// every element cost more than the arithmetic they choose).
template <typename T, int ELEMS, int GATE, bool BWD>
__global__ void __launch_bounds__(512) gated_norm_kernel(const GatedArgs a, int tpr, int rpb, int parts)
{
    constexpr int E = Vec<T>::N, NV = ELEMS / E;
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
    Raw<T, NV, E> xr, zr, dr;   // of the next row
    auto fetch = [&](int64_t r0) {
        const bool live = r0 + sub < a.rows;
        const int64_t base = live ? (r0 + sub) * a.dim + col : 0;
        xr.load(x + base, lane_r, tpr, in, live);
        if (GATE)
            zr.load(z + base, lane_r, tpr, in, live);
        if (BWD)
            dr.load(dout + base, lane_r, tpr, in, live);
    };
    const int64_t stride = (int64_t)parts * rpb;
    fetch((int64_t)part * rpb);
    // every thread of the block takes the same number of turns (barriers)
    for (int64_t r0 = (int64_t)part * rpb; r0 < a.rows; r0 += stride) {
        const bool live = r0 + sub < a.rows;
        const int64_t base = (r0 + sub) * a.dim + col;
        float xv[NV][E], zv[NV][E], dv[NV][E];
        xr.get(xv);
        if (GATE)
            zr.get(zv);
        if (BWD)
            dr.get(dv);
        if (r0 + stride < a.rows)
            fetch(r0 + stride);
        float sg[NV][E];   // sigmoid(z)
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int e = 0; e < E; e++) {
                sg[v][e] = GATE ? sigmoid_mufu(zv[v][e]) : 1.f;
                const float s = GATE ? zv[v][e] * sg[v][e] : 1.f;
                const float u = GATE == 1 ? xv[v][e] * s : xv[v][e];
                sum[0] = fmaf(u, u, sum[0]);
                if (BWD)
                    sum[1] = fmaf((GATE == 2 ? dv[v][e] * s : dv[v][e]) * w[v][e], u, sum[1]);
            }
        if (BWD) {
            row_sum<2>(sum, tpr, red, turn);
        } else {
            float one[1] = {sum[0]};
            row_sum<1>(one, tpr, red, turn);
            sum[0] = one[0];
        }
        // behind the last row 0, so that eps = 0 leaves no 0 / 0 in dw
        const float r = live ? rsqrtf(sum[0] * inv + a.eps) : 0.f;
        const float m = sum[1] * inv * r;   // mean(dn n)
#pragma unroll
        for (int v = 0; v < NV; v++) {
            const int64_t at = base + (lane_r + v * tpr) * E;
            float o[E], oz[E];
#pragma unroll
            for (int e = 0; e < E; e++) {
                const float zz = GATE ? zv[v][e] : 0.f, s = GATE ? zz * sg[v][e] : 1.f;
                const float n = (GATE == 1 ? xv[v][e] * s : xv[v][e]) * r;
                if (!BWD) {
                    o[e] = GATE == 2 ? n * w[v][e] * s : n * w[v][e];
                } else {
                    const float ds = GATE ? sg[v][e] * fmaf(zz, 1.f - sg[v][e], 1.f) : 0.f;
                    const float dy = GATE == 2 ? dv[v][e] * s : dv[v][e];
                    dw[v][e] = fmaf(dy, n, dw[v][e]);
                    const float du = r * fmaf(-n, m, dy * w[v][e]);
                    o[e] = GATE == 1 ? du * s : du;
                    oz[e] = (GATE == 2 ? dv[v][e] * n * w[v][e] : du * xv[v][e]) * ds;
                }
            }
            if (live && in[v]) {
                store_row<T, E>(static_cast<T *>(BWD ? a.dx : a.out) + at, o);
                if (BWD && GATE)
                    store_row<T, E>(static_cast<T *>(a.dz) + at, oz);
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

// parts: how many blocks shared the rows of a group (for the column sums)
template <typename T, bool BWD> cudaError_t launch_typed(const GatedArgs &a, cudaStream_t st, int *parts)
{
    const NormPlan p = norm_threads(a.group);
    const int G = a.dim / a.group;
    const size_t smem = BWD ? a.group * sizeof(float) : 0;
    auto go = [&](auto kernel) {
        *parts = (int)parts_for(a.rows, G, p, resident_blocks(kernel, p.threads, smem));
        kernel<<<(unsigned)(*parts * G), p.threads, smem, st>>>(a, p.tpr, p.rows_at_once, *parts);
    };
    if (!a.z)
        p.elems == 8 ? go(gated_norm_kernel<T, 8, 0, BWD>) : go(gated_norm_kernel<T, 16, 0, BWD>);
    else if (!a.norm_first)
        p.elems == 8 ? go(gated_norm_kernel<T, 8, 1, BWD>) : go(gated_norm_kernel<T, 16, 1, BWD>);
    else
        p.elems == 8 ? go(gated_norm_kernel<T, 8, 2, BWD>) : go(gated_norm_kernel<T, 16, 2, BWD>);
    return cudaGetLastError();
}

struct Sums {
    PartSum s[kMaxSums];
};
// Block: 32 columns x 32 strands of the partial rows of one sum and set; the
// strands are joined in order.
__global__ void __launch_bounds__(1024) part_sum_kernel(const Sums sums, int dim)
{
    __shared__ float s[32][33];
    const PartSum &j = sums.s[blockIdx.z];
    const int c = blockIdx.x * 32 + threadIdx.x;
    for (int64_t set = blockIdx.y; set < j.sets; set += gridDim.y) {
        const float *p = j.parts + (size_t)set * j.nparts * dim;
        float v = 0.f;
        if (c < dim)
            for (int k = threadIdx.y; k < j.nparts; k += 32)
                v += p[(size_t)k * dim + c];
        s[threadIdx.y][threadIdx.x] = v;
        __syncthreads();
        // warp y sums column y of the block over the strands
        const float t = warp_sum(s[threadIdx.x][threadIdx.y]);
        const int col = blockIdx.x * 32 + threadIdx.y;
        if (threadIdx.x == 0 && col < dim)
            j.out[(size_t)set * dim + col] = t;
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_part_sums(const PartSum *sums, int n, int dim, cudaStream_t st)
{
    Sums j;
    int64_t most = 1;
    for (int k = 0; k < n; k++) {
        j.s[k] = sums[k];
        most = sums[k].sets > most ? sums[k].sets : most;
    }
    const dim3 grid((dim + 31) / 32, (unsigned)(most < 65535 ? most : 65535), n);
    part_sum_kernel<<<grid, dim3(32, 32), 0, st>>>(j, dim);
    return cudaGetLastError();
}

size_t gated_bwd_workspace(int64_t rows, int dim, int group)
{
    const NormPlan p = norm_threads(group);
    return (size_t)parts_for(rows, dim / group, p, (int64_t)kSMs * (2048 / p.threads)) * dim * sizeof(float);
}

cudaError_t launch_gated_fwd(const GatedArgs &a, cudaStream_t st)
{
    int parts;
    return a.dtype == 0 ? launch_typed<float, false>(a, st, &parts) : launch_typed<__nv_bfloat16, false>(a, st, &parts);
}

cudaError_t launch_gated_bwd(const GatedArgs &a, cudaStream_t st)
{
    int parts = 0;
    const cudaError_t e =
        a.dtype == 0 ? launch_typed<float, true>(a, st, &parts) : launch_typed<__nv_bfloat16, true>(a, st, &parts);
    if (e != cudaSuccess)
        return e;
    const PartSum sum{a.parts, a.dweight, 1, parts};
    return launch_part_sums(&sum, 1, a.dim, st);
}

}  // namespace ssm
