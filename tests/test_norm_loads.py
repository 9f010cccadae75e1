"""Which loads the layer norm and dropout kernels use.  An [M,N] output may be one of the inputs, so
no [M,N] tensor goes through the read-only path (ld.global.nc, __ldg), which is defined for memory
that the kernel does not write.  No run can show it: each element is read and written by one thread."""
import os
import re

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "quantize_fp8_gemm_gb300", "csrc")


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//.*", "", f.read())


def test_tensors_that_may_be_outputs_are_not_read_through_the_read_only_path():
    read_only = {m.group(1) for m in re.finditer(r"(\w+)\([^()]*\)\s*\{[^}]*ld\.global\.nc", text("common.cuh"))}
    assert "ld_stream_v4" in read_only  # what the quantize kernels use: their outputs are never their inputs
    names = sorted(n for n in os.listdir(CSRC) if n.startswith(("norm_", "dropout")))
    assert "norm_ops.cuh" in names and "dropout.cu" in names
    for name in names:
        src = text(name)
        for fn in read_only:
            assert not re.search(rf"\b{fn}\b", src), f"{name} uses {fn}"
        assert "ld.global.nc" not in src and "__restrict__" not in src, name
        # the parameter vectors alone
        assert re.sub(r"load_params2\(.*?\n}\n", "", src, flags=re.S).count("__ldg") == 0, name
