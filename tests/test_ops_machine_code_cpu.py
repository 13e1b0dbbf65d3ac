"""What the 8-bit product's code rests on in the compiler, seen in gfx950 assembly of its own
functions (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

from fp32_gemm_f32_amd import build

pytestmark = pytest.mark.skipif(
    shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not available")

PROBE = """
#include "kernel_i8.hpp"
__global__ void value(float *c, const int *sum, const float *s)
{
    c[0] = sgemm::i8_value(sum[0], s[0], s[1], s[2]);
}
"""


def test_scaling_and_bias_share_one_rounding(tmp_path):
    """i8_value is a fused multiply-add by its own wording: the compiler has no say in it."""
    src, out = tmp_path / "value.hip", tmp_path / "value.s"
    src.write_text(PROBE)
    subprocess.run([build.hipcc(), *build.flags(False), "-ffp-contract=off", "--cuda-device-only", "-S", str(src),
                    "-o", str(out)], check=True, capture_output=True)
    text = out.read_text()
    code = text[text.index("_Z5valuePfPKiPKf:"):]
    code = code[:code.index("s_endpgm")]
    assert "v_fma" in code and "v_add_f32" not in code, code


NARROW = """
#include "kernel_i8.hpp"
__global__ void narrow(_Float16 *c, const int *sum, const float *s)
{
    c[threadIdx.x] = sgemm::Elem<SGEMM_DTYPE_F16>::narrow(sgemm::i8_value(sum[threadIdx.x], s[0], s[1], s[2]));
}
"""


def test_fp16_results_are_rounded_to_fp32_first(tmp_path):
    """No instruction that multiplies, adds and rounds to FP16 in one: it would give other bits than
    kernels in which the compiler does not find it."""
    src, out = tmp_path / "narrow.hip", tmp_path / "narrow.s"
    src.write_text(NARROW)
    subprocess.run([build.hipcc(), *build.flags(False), "--cuda-device-only", "-S", str(src), "-o", str(out)],
                   check=True, capture_output=True)
    text = out.read_text()
    code = text[text.index("_Z6narrowPDF16_PKiPKf:"):]
    code = code[:code.index("s_endpgm")]
    assert "mix" not in code and "v_cvt_f16_f32" in code, code
