// block_norm_fp16.cu -- the one-pass kernels of block_norm_fwd and block_norm_bwd for fp16, rows on the 16-byte grid.
#include "block_norm.cuh"

template cudaError_t fp8q::launch_bn_fwd<__half, false>(const BnFwd<__half>&, cudaStream_t);
template cudaError_t fp8q::launch_bn_bwd<__half, false, false>(const BnBwd<__half>&, int, int*, cudaStream_t);
template cudaError_t fp8q::launch_bn_bwd<__half, true, false>(const BnBwd<__half>&, int, int*, cudaStream_t);
