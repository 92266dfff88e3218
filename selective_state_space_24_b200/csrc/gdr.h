// gdr.h -- launcher interface of the gated delta rule kernels.  Not part of
// the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssm {

struct GdrArgs {
    int Bsz, L, Hk, Hv, K, V;
    int dtype;                       // 0 = float32, 1 = bf16
    int softplus, sigmoid, l2norm;
    float scale;
    const void *q, *k, *v, *delta, *beta;
    const float *bias, *A;
    const float *init;               // (B, Hv, V, K) or nullptr
    void *out;
    float *last;                     // (B, Hv, V, K) or nullptr
    void *workspace;
    unsigned wait_limit;             // gdr_stall_set's, of a call that is to stall
    int withhold_chunk;
};

// Step by step, the state in registers: one token (gdr_step) or short
// sequences.
cudaError_t launch_gdr_recurrent(const GdrArgs &a, cudaStream_t st);

cudaError_t launch_gdr_chunk(const GdrArgs &a, cudaStream_t st);
// Test setting of the chunked forward kernel's bounded waits (process-wide):
// the chunk to withhold (< 0: none) and the waits' limit (0: the default).
void gdr_stall_set(int withhold_chunk, unsigned wait_limit);
// The kernels' device-side error word (a bounded wait that gave up).
cudaError_t read_and_clear_gdr_error(unsigned *value, cudaStream_t stream);

struct GdrBwdArgs {
    GdrArgs f;
    const void *dout;
    const float *dlast;              // or nullptr
    void *dq, *dk, *dv, *ddelta, *dbeta;
    float *dA, *dbias, *dinit;       // dbias, dinit may be nullptr
};
size_t gdr_bwd_ws_bytes(const GdrArgs &a);
cudaError_t launch_gdr_bwd(const GdrBwdArgs &a, cudaStream_t st);

}  // namespace ssm
