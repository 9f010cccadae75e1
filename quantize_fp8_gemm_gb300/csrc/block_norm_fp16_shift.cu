// block_norm_fp16_shift.cu -- the one-pass kernels of block_norm_fwd and block_norm_bwd for fp16, rows off the 16-byte grid.
#include "block_norm.cuh"

template cudaError_t fp8q::launch_bn_fwd<__half, true>(const BnFwd<__half>&, cudaStream_t);
template cudaError_t fp8q::launch_bn_bwd<__half, false, true>(const BnBwd<__half>&, int, int*, cudaStream_t);
template cudaError_t fp8q::launch_bn_bwd<__half, true, true>(const BnBwd<__half>&, int, int*, cudaStream_t);
