"""CPU checks of how paged_attention shares out its work, as far as the size of
its workspace shows it: 0 where blocks take whole units, 8 bytes of maximum and
sum and the fp32 row for each row of the parts that cut units leave otherwise."""
import pytest

import bit_gemv_amd as bg


def _need(rows, q_heads, heads, d, b, room, max_rows, max_kv):
    return bg.load_library().paged_attention_workspace_bytes(rows, q_heads, heads, d, b, room // 16, 16, max_rows, max_kv)


def _parts(blocks, heads, row_tile, d):
    return 2 * blocks * heads * row_tile * (d + 2) * 4


@pytest.mark.parametrize("chunk,own", [(300, _parts(32, 8, 256, 128)), (2000, 0), (20000, 0)])
def test_single_tokens_beside_a_chunk_are_cut_as_they_are_alone(chunk, own):
    """Three long single tokens beside a prompt (own: what the prompt's launch
    needs): too few units for the kernel to take them whole, however long the
    prompt is. Blocks of the single tokens' launch: one for each step of 128
    tokens that its sequences can hold, up to 512 over the key heads."""
    kv = max(2000, chunk)
    steps = 4 * ((kv + 127) // 128)
    assert _need(chunk + 3, 64, 8, 128, 4, 32768, chunk, kv) == own + _parts(min(64, steps), 8, 16, 128)


def test_groups_without_a_place_among_few_rows_take_one_launch():
    """A group of more than 16 heads has no sequence of up to 16 query rows."""
    d = 64
    one = _need(306, 40, 2, d, 7, 8192, 300, 8192)
    assert one == _parts(256, 2, 128, d)
