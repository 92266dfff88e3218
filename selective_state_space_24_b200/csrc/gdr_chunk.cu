// gdr_chunk.cu -- the gated delta rule over sequences.
#include "gdr_math.cuh"

namespace ssm {

size_t gdr_chunk_ws_bytes(const GdrArgs &) { return 0; }

cudaError_t launch_gdr_chunk(const GdrArgs &a, cudaStream_t st) { return launch_gdr_recurrent(a, st); }

}  // namespace ssm
