// norm_fwd_fp32_shift.cu -- layer_norm_fwd's one-pass kernels for fp32, rows off the 16-byte grid.
#include "norm_fwd.cuh"

template cudaError_t fp8q::launch_fwd_ring<float, true>(const FwdParams<float>&, cudaStream_t);
