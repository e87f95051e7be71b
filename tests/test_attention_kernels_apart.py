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


def _few(kernels, d, bits, sym):
    """(streaming keys, text) of the kernels for few rows of a format"""
    name = re.compile(f"attn_few_kernelILi{d}ELi{bits}ELb{int(sym)}ELi\\d+ELi\\d+ELb([01])ELb0E")
    return [(m[1] == "1", text) for n, text in kernels.items() if (m := name.search(n))]


@pytest.mark.parametrize("d,bits,sym", [(d, b, s) for d in (64, 128, 256) for b in (4, 8) for s in (False, True)])
def test_keys_come_by_streaming_loads(kernels, d, bits, sym):
    """Every format has kernels whose keys and values come by streaming loads, and
    only asymmetric INT8 of 128-wide heads, where both ways were measured to win,
    has them with ordinary loads of the keys as well."""
    both = (d, bits, sym) == (128, 8, False)
    found = _few(kernels, d, bits, sym)
    assert sorted(s for s, _ in found) == ([False, False] if both else []) + [True, True]
    words = d * bits // 128                           # code words a lane and 16 keys, up to 4 a load
    of_side = 2 * max(1, words // 4)                  # loads of a tile's keys, or of its values
    load = f"global_load_dwordx{min(words, 4)} .* nt$"
    for stream, text in found:
        n = len(re.findall(load, text, re.M))
        # as often as a tile is loaded in the text; without the keys' half as many
        assert n > 0 and n % of_side == 0, n
        if both:
            most = max(len(re.findall(load, t, re.M)) for _, t in found)
            assert (n == most) == stream and (stream or 2 * n <= most), (n, most)
