// norm_fwd_fp16_shift.cu -- layer_norm_fwd's one-pass kernels for fp16, rows off the 16-byte grid.
#include "norm_fwd.cuh"

template cudaError_t fp8q::launch_fwd_ring<__half, true>(const FwdParams<__half>&, cudaStream_t);
