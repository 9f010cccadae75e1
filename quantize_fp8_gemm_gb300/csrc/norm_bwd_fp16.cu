// norm_bwd_fp16.cu -- layer_norm_bwd's one-pass kernels for fp16.
#include "norm_bwd.cuh"

template cudaError_t fp8q::launch_bwd_ring<__half, false>(BwdParams<__half>&, cudaStream_t);
template cudaError_t fp8q::launch_bwd_ring<__half, true>(BwdParams<__half>&, cudaStream_t);
