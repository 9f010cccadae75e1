// block_norm_bf16_shift.cu -- the one-pass kernels of block_norm_fwd and block_norm_bwd for bf16, rows off the 16-byte grid.
#include "block_norm.cuh"

template cudaError_t fp8q::launch_bn_fwd<__nv_bfloat16, true>(const BnFwd<__nv_bfloat16>&, cudaStream_t);
template cudaError_t fp8q::launch_bn_bwd<__nv_bfloat16, false, true>(const BnBwd<__nv_bfloat16>&, int, int*, cudaStream_t);
template cudaError_t fp8q::launch_bn_bwd<__nv_bfloat16, true, true>(const BnBwd<__nv_bfloat16>&, int, int*, cudaStream_t);
