// The gradients of the block norms for CTAs of 512 threads (norm_bwd.cuh).
#include "norm_bwd.cuh"

int moe::block_norm_bwd_512(NormBwd p, int dtype, int grad_dtype, int* parts, cudaStream_t st) {
  return bwd_typed<kWideThreads>(p, dtype, grad_dtype, parts, st);
}
