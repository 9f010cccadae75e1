"""quantize_fp8_gemm_gb300 -- the forward FP8 MLP down-projection on one GB300.

The compute lives in libfp8q.so (hand-written sm_103a CUDA behind the C ABI of
include/fp8q.h).  This package is its Python face:

* ``binding``   -- ctypes wrappers with the C names (fp8_quant_fused,
                   fp8_gemm_fwd, fp8_gemm_dgrad, amax_history_update,
                   layer_norm_fwd, dropout_fwd, fp8_glu_fwd, block_norm_fwd), taking torch CUDA tensors for
                   device memory and the current stream.
* ``downproj``  -- the call order and buffers of one training step with
                   delayed per-tensor (or 1x128 / 128x128 group) scales.
* ``mlpstack``  -- whole MLP sub-layers, forward and backward: layer norm,
                   dropout and residual around the FP8 GEMMs.
* ``gatedstack`` -- gated MLP sub-layers with norms before and after the block,
                   a gate and a residual scale, forward and backward.
* ``workloads`` -- seeded synthetic inputs of the benchmark workloads.
* ``build``     -- nvcc build of libfp8q.so, in-tree.

Importing the package does not load the library; the first call does, and
raises if it has not been built.
"""
from .binding import (ACT_GELU, ACT_IDENTITY, ACT_RELU, ACT_RELU2, ACT_SILU, DEV_BAD_AMAX, DEV_TIMEOUT, E4M3, E5M2,
                      GROUP, Fp8qError, amax_history_update, block_norm_bwd, block_norm_bwd_workspace_bytes,
                      block_norm_fwd, dropout_bwd, dropout_fwd, fp8_gemm_dgrad, fp8_gemm_dgrad_glu, fp8_gemm_fwd, fp8_glu_fwd,
                      fp8_quant_fused, fp8q_naive_act, fp8q_naive_amax, fp8q_naive_cast, layer_norm_bwd,
                      layer_norm_bwd_workspace_bytes, layer_norm_fwd)
from .downproj import DelayedScale, Fp8DownProj
from .gatedstack import Fp8GatedMlpStack
from .mlpstack import Fp8MlpStack

__all__ = [
    "ACT_GELU", "ACT_IDENTITY", "ACT_RELU", "ACT_RELU2", "ACT_SILU", "DEV_BAD_AMAX", "DEV_TIMEOUT", "E4M3", "E5M2", "GROUP",
    "Fp8qError", "amax_history_update", "dropout_bwd", "dropout_fwd", "fp8_gemm_dgrad", "fp8_gemm_fwd",
    "fp8_quant_fused", "fp8q_naive_act", "fp8q_naive_amax", "fp8q_naive_cast", "layer_norm_bwd",
    "layer_norm_bwd_workspace_bytes", "layer_norm_fwd", "DelayedScale", "Fp8DownProj",
    "Fp8MlpStack", "Fp8GatedMlpStack", "block_norm_bwd", "block_norm_bwd_workspace_bytes", "block_norm_fwd",
    "fp8_gemm_dgrad_glu", "fp8_glu_fwd",
]
