"""The line that bench.py prints: all that its readers need, and no longer than a log's last 3000 characters hold."""
import json
import sys

from tests.conftest import ROOT

sys.path.insert(0, ROOT)
import bench  # noqa: E402
from quantize_fp8_gemm_gb300 import workloads as WL  # noqa: E402


def record():
    """A run's record on the largest workload, with figures of full length and texts as the run writes them."""
    w, f = WL.WORKLOADS["gpt2xl"], 1234.567890123456
    peaks, fp8 = {"hbm_gbs": 6791.7, "source": "measured"}, {"tflops": 3823.6, "source": "x" * 80, "cublaslt_e4m3_8192_tflops": f}
    kern = {k: 0.123456789012345678 for k in ("quant", "gemm", "fused_step_kernel", "step", "history")}
    roof = bench.rooflines(w, kern, peaks, fp8, "gpt2xl", step_ms=1.0512345678901234)
    roof["dominant"]["traffic"] = 4220518400.0
    cpu = {"value": 0.0191234567890123, "unit": "TFLOP/s", "cores": 144, "kind": "oracle", "quant_gbs": f, "quant_s": f,
           "gemm_ms_per_row": f, "gemm_full_extrapolated_s": f, "sample": "x" * 330}
    return {
        "metric": bench.METRIC, "value": f, "unit": bench.UNIT, "n_gpus": 8, "steps": 200, "warmup": 10, "ms_per_step": f,
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "e4m3 x e4m3 -> f32 accumulate -> bf16",
        "data": "synthetic (seeded numpy normals rounded to BF16, uploaded before timing)",
        "config": {"workload": w.name, "M": w.M, "K": w.K, "N": w.N, "act": "relu2", "scaling": "per-tensor delayed", "margin": 2.0,
                   "history": 1, "l2": "flushed before every step (256 MiB write + read, untimed)", "step": "x" * 150},
        "kernel_ms": kern, "quant_hbm_gbs": f, "gemm_tflops": f, "roofline": roof["dominant"], "roofline_quant": roof["quant"],
        "roofline_gemm": roof["gemm"], "roofline_fused": roof["fused"], "fp8_peak": fp8, "cpu_baseline": cpu,
        "e2e": {"value": f, "unit": "TFLOP/s", "h2d_bytes_per_step": 1698201600, "d2h_bytes_per_step": 419430400, "ms_per_step": f,
                "steps": 200, "schedule": "x" * 90},
        "gpu_launches": 200, "kernel_ms_note": "x" * 150, "timing": "x" * 90,
        "clocks": {"sm_mhz": 1995.0, "sm_max_mhz": 2070.0, "reasons": ["sw_power_cap", "hw_slowdown"], "samples": 100},
        "wall_s_timed_loop": f, "extras": {f"row {i}": {"shape": "x" * 60, "ms": f} for i in range(100)},
    }


def test_the_printed_line_is_short_and_whole():
    line = record()
    got = bench.printed_line(line)
    assert len(json.dumps(got)) <= 2800
    for k in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling", "vs_baseline",
              "dtype", "data", "config", "e2e", "gpu_launches", "clocks", "cpu_baseline"):
        assert got[k] == line[k], k
    assert {"kernel", "achieved", "peak", "unit", "frac", "traffic"} <= set(got["roofline"])
    assert "extras" not in got and len(json.dumps(line)) > 8000
