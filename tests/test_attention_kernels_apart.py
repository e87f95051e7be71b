"""CPU checks of the attention kernels that paged_attention is compiled to: they
are its own, without the forms of cross_attention and prefix_attention, which
cost it up to 1.7 % where they were looked at on the device."""
import os
import re
import subprocess

import pytest

from bit_gemv_amd import build

pytestmark = [pytest.mark.slow, pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """name -> text of each kernel of attention.hip over rows and keys"""
    out = tmp_path_factory.mktemp("attention") / "attention.s"
    subprocess.run([build.HIPCC, *build.CXXFLAGS, *build.EXTRA["attention.hip"], "--cuda-device-only", "-S",
                    os.path.join(build.CSRC, "attention.hip"), "-o", str(out)], check=True, capture_output=True)
    found = re.findall(r"^(_ZN\S*attn_(?:few|many)_kernel\S*):[^\n]*\n(.*?)^\.Lfunc_end", out.read_text(), re.S | re.M)
    return dict(found)


def test_paged_attention_has_no_forms_beside_its_own(kernels):
    assert len(kernels) >= 24 + 20                    # 8- and 16-row tiles of three widths and four formats; many rows
    for name in kernels:
        assert name.endswith("ELb0EEEvNS_8AttnArgsENS0_4SpanE"), name    # their last argument of the template
