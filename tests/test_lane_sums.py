"""The exchange that adds sixteen values over the lanes of a row, compiled for the GPU and read as assembly (CPU)."""
import os
import re
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

KERNEL = """
#include "wave.hpp"
extern "C" __global__ void k(const float *in, float *out)
{
    float x[16];
    for (int i = 0; i < 16; ++i)
        x[i] = in[i %% %d * 64 + threadIdx.x];
    out[threadIdx.x] = chol::over_lanes(x, threadIdx.x);
}
"""


@pytest.mark.parametrize("different", [16, 8, 4, 1])
def test_results_share_no_register_with_operands(tmp_path, different):
    """Values that are equal (here by where they come from) may not meet in one register: results are written before
    the last operand is read."""
    build = pytest.importorskip("differentiable_cholesky_amd.build")
    source, out = tmp_path / "k.hip", tmp_path / "k.txt"
    source.write_text(KERNEL % different)
    subprocess.run([build.HIPCC, *build.FLAGS, "-I", build.CSRC, "--offload-device-only", "-S", str(source), "-o", str(out)],
                   check=True, capture_output=True, timeout=120)
    first = re.findall(r"v_add_f32_dpp (v\d+), (v\d+), (v\d+) row_ror:8 row_mask:0xf bank_mask:(\w+)", out.read_text())
    assert len(first) == 16 and all(a == b for _, a, b, _ in first)
    results = {d for d, _, _, _ in first}
    operands = {s for _, s, _, mask in first if mask == "0xc"}
    assert len(results) == 8 and not results & operands, first
