// block_norm_fp32.cu -- the one-pass kernels of block_norm_fwd and block_norm_bwd for fp32, rows on the 16-byte grid.
#include "block_norm.cuh"

template cudaError_t fp8q::launch_bn_fwd<float, false>(const BnFwd<float>&, cudaStream_t);
template cudaError_t fp8q::launch_bn_bwd<float, false, false>(const BnBwd<float>&, int, int*, cudaStream_t);
template cudaError_t fp8q::launch_bn_bwd<float, true, false>(const BnBwd<float>&, int, int*, cudaStream_t);
