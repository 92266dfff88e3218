// norm.h -- launcher interface of the norm kernels.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssm {

// How threads cover rows (of one group of columns): tpr threads per row, a
// power of two, each holding `elems` elements; a block works on threads / tpr
// rows at a time.  Block b owns the columns of group b % G and walks rows
// with a stride, so a thread's columns never change: its weights stay in
// registers and column sums gather there.  Several blocks share the rows of
// one group (or sample), each with a partial sum of its own.
struct NormPlan {
    int elems, tpr, threads;
    int rows_at_once;   // rows a block works on at a time
};

struct GatedArgs {
    int64_t rows;          // of `dim` elements
    int dim, group;
    float eps;
    int dtype, norm_first;
    const void *x, *z, *dout;
    const float *weight;
    void *out, *dx, *dz;
    float *dweight, *parts;   // parts: (parts, dim)
};
size_t gated_bwd_workspace(int64_t rows, int dim, int group);
cudaError_t launch_gated_fwd(const GatedArgs &a, cudaStream_t st);
cudaError_t launch_gated_bwd(const GatedArgs &a, cudaStream_t st);

struct ResidualArgs {
    int64_t rows, samples;
    int dim;
    float eps, alpha;
    float fdim;                // dim (read as a constant, it takes no register: 9 blocks per SM, not 8)
    int dtype, layer, res32;   // res32: the stream is float32
    const void *x, *residual, *dout, *dres_out;
    const float *weight, *bias, *scale, *post;
    void *res_out, *out, *dx, *dres;
    float *dweight, *dbias, *dscale, *dpost, *parts;
};
size_t residual_bwd_workspace(int64_t rows, int64_t samples, int dim, bool has_bias, bool has_scale,
                              bool has_post);
cudaError_t launch_residual_fwd(const ResidualArgs &a, cudaStream_t st);
cudaError_t launch_residual_bwd(const ResidualArgs &a, cudaStream_t st);

// Sums of partial rows, several at once: out[s][c] = sum over p < nparts of
// parts[s][p][c] for s < sets, in a fixed order.
struct PartSum {
    const float *parts;
    float *out;
    int64_t sets;
    int nparts;
};
constexpr int kMaxSums = 4;
cudaError_t launch_part_sums(const PartSum *sums, int n, int dim, cudaStream_t st);

}  // namespace ssm
