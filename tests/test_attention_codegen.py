"""CPU check of the compiled attention kernels: the many-row kernels' weights
(exponentials) stand beside matrix instructions, in every format. The compiler
once moved the asymmetric formats' out of that run of instructions, which no
result shows."""
import os
import re
import subprocess

import pytest

from bit_gemv_amd import build

pytestmark = [pytest.mark.slow, pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")]


def _many_row_kernels(asm):
    """(name, text) of each"""
    return re.findall(r"^(_ZN\S*attn_many_kernel\S*):[^\n]*\n(.*?)^\.Lfunc_end", asm, re.S | re.M)


def test_weights_stand_beside_the_products(tmp_path):
    out = tmp_path / "attention.s"
    subprocess.run([build.HIPCC, *build.CXXFLAGS, *build.EXTRA["attention.hip"], "--cuda-device-only", "-S",
                    os.path.join(build.CSRC, "attention.hip"), "-o", str(out)], check=True, capture_output=True)
    kernels = _many_row_kernels(out.read_text())
    assert len(kernels) == 20                        # 64 and 128 wide: 128 and 256 rows; 256 wide: 128; four formats
    for name, text in kernels:
        runs = [b for b in re.split(r"^\.LBB\S*:", text, flags=re.M) if "v_mfma" in b]
        beside = sum(len(re.findall("v_exp_f32", b)) for b in runs)
        assert beside >= 32, (name, beside)          # 16 for each of a tile's two blocks at least
