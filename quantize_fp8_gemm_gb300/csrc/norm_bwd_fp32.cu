// norm_bwd_fp32.cu -- layer_norm_bwd's one-pass kernels for fp32.
#include "norm_bwd.cuh"

template cudaError_t fp8q::launch_bwd_ring<float, false>(BwdParams<float>&, cudaStream_t);
template cudaError_t fp8q::launch_bwd_ring<float, true>(BwdParams<float>&, cudaStream_t);
