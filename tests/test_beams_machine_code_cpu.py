"""What the beam step's sums rest on in the compiler, seen in gfx950 assembly of their own function (no
GPU needed)."""
import os
import shutil
import subprocess

import pytest

from fp32_gemm_f32_amd import build

pytestmark = pytest.mark.skipif(
    shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not available")

PROBE = """
#include "kernel_beams.hpp"
__global__ void rescale(float *p)
{
    sgemm::BeamStats st;
    st.m = p[threadIdx.x];
    st.s = p[64 + threadIdx.x];
    st.raise(p[128 + threadIdx.x]);
    p[threadIdx.x] = st.m;
    p[64 + threadIdx.x] = st.s;
}
"""


def test_both_references_are_rounded(tmp_path):
    """A sum is taken over a rounded reference; raising it to another one subtracts two rounded products,
    with no multiply-add that keeps one of them whole."""
    src, out = tmp_path / "rescale.hip", tmp_path / "rescale.s"
    src.write_text(PROBE)
    subprocess.run([build.hipcc(), *build.flags(True), "--cuda-device-only", "-S", str(src), "-o", str(out)],
                   check=True, capture_output=True)
    text = out.read_text()
    code = text[text.index("_Z7rescalePf:"):]
    code = code[:code.index("s_endpgm")]
    assert "v_exp_f32" in code and "v_sub_f32" in code
    assert "v_fma" not in code and "v_mad" not in code and "v_mac" not in code and "v_fmac" not in code, code
