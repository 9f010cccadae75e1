"""The launch table of the layer norm and dropout kernels (csrc/launch_table.cuh): what it keeps is
one device's.  Host C++, compiled and run here; no GPU."""
import os
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "quantize_fp8_gemm_gb300", "csrc")

PROGRAM = r"""
#include "launch_table.cuh"
#include <cstdio>
enum Error { kOk = 0, kFailed = 7 };
static fp8q::DeviceTable<17> table;
static int asked = 0;
#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
int main() {
    auto answer = [](int v, Error e = kOk) { return [v, e](int* n) { ++asked; *n = v; return e; }; };
    int n = 0;
    CHECK(table.get(0, 4, &n, answer(3)) == kOk && n == 3 && asked == 1);
    CHECK(table.get(0, 4, &n, answer(9)) == kOk && n == 3 && asked == 1);   // kept
    CHECK(table.get(0, 16, &n, answer(1)) == kOk && n == 1 && asked == 2);  // another size
    CHECK(table.get(1, 4, &n, answer(2)) == kOk && n == 2 && asked == 3);   // another device is asked itself
    CHECK(table.get(1, 4, &n, answer(9)) == kOk && n == 2 && asked == 3);
    CHECK(table.get(0, 4, &n, answer(9)) == kOk && n == 3 && asked == 3);
    CHECK(table.get(2, 4, &n, answer(5, kFailed)) == kFailed && asked == 4);  // an error is returned, not kept
    CHECK(table.get(2, 4, &n, answer(5)) == kOk && n == 5 && asked == 5);
    for (int i = 0; i < 2; ++i)  // past the table: asked every time
        CHECK(table.get(fp8q::kMaxDevices, 4, &n, answer(6)) == kOk && n == 6 && asked == 6 + i);
    CHECK(table.get(fp8q::kMaxDevices - 1, 16, &n, answer(4)) == kOk && n == 4 && asked == 8);
    return 0;
}
"""


def test_kept_by_device_and_size(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "table.cpp", tmp_path / "table"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout


def test_launchers_keep_nothing_beside_it():
    """No launcher of these kernels has a table of its own, which would hold for every device."""
    for name in ("norm_fwd.cuh", "norm_bwd.cuh", "norm_fwd.cu", "norm_bwd.cu", "dropout.cu"):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        assert "static std::" not in text and "static int" not in text, name
