// norm_fwd_bf16.cu -- layer_norm_fwd's one-pass kernels for bf16, rows on the 16-byte grid.
#include "norm_fwd.cuh"

template cudaError_t fp8q::launch_fwd_ring<__nv_bfloat16, false>(const FwdParams<__nv_bfloat16>&, cudaStream_t);
