// block_norm_bf16.cu -- the one-pass kernels of block_norm_fwd and block_norm_bwd for bf16, rows on the 16-byte grid.
#include "block_norm.cuh"

template cudaError_t fp8q::launch_bn_fwd<__nv_bfloat16, false>(const BnFwd<__nv_bfloat16>&, cudaStream_t);
template cudaError_t fp8q::launch_bn_bwd<__nv_bfloat16, false, false>(const BnBwd<__nv_bfloat16>&, int, int*, cudaStream_t);
template cudaError_t fp8q::launch_bn_bwd<__nv_bfloat16, true, false>(const BnBwd<__nv_bfloat16>&, int, int*, cudaStream_t);
