// norm_bwd_bf16.cu -- layer_norm_bwd's one-pass kernels for bf16.
#include "norm_bwd.cuh"

template cudaError_t fp8q::launch_bwd_ring<__nv_bfloat16, false>(BwdParams<__nv_bfloat16>&, cudaStream_t);
template cudaError_t fp8q::launch_bwd_ring<__nv_bfloat16, true>(BwdParams<__nv_bfloat16>&, cudaStream_t);
