"""CPU checks of how paged_attention shares out its work, as far as the size of
its workspace shows it: 0 where blocks take whole units, 8 bytes of maximum and
sum and the fp32 row for each row of the parts that cut units leave otherwise."""
import random

import pytest

import bit_gemv_amd as bg
from attention_forms import forms


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


@pytest.mark.parametrize("b,heads,whole", [(16, 8, False), (64, 2, False), (32, 8, True), (8, 32, True)])
def test_decode_batches_of_up_to_2048_tokens_are_whole_where_units_fill_the_card(b, heads, whole):
    assert (_need(b, 8 * heads, heads, 128, b, 2048, 1, 2000) == 0) == whole


def test_groups_without_a_place_among_few_rows_take_one_launch():
    """A group of more than 16 heads has no sequence of up to 16 query rows."""
    d = 64
    one = _need(306, 40, 2, d, 7, 8192, 300, 8192)
    assert one == _parts(256, 2, 128, d)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_the_model_of_the_forms_is_the_librarys(d):
    """attention_forms.forms, by which the GPU tests name the form they reach,
    checks its workspace against the library's: ragged batches, exact, loose,
    small and missing hints."""
    rng = random.Random(d)
    seen = set()
    for _ in range(400):
        heads, group, b = rng.choice([1, 2, 5, 8, 32, 64]), rng.choice([1, 2, 3, 7, 8, 16, 20]), rng.choice([1, 2, 4, 9, 70, 300])
        seqs = []
        for _ in range(b):
            n = rng.choice([0, 1, 1, 1, 1, 2, 40, rng.randrange(1, 600)])
            seqs.append((n + rng.choice([0, 5, 700, rng.randrange(5000)]), n))
        rows = sum(n for _, n in seqs) + rng.randrange(2)
        if rows == 0:
            continue
        most, room = max(n for _, n in seqs), 16 * rng.choice([400, 700, 4096])
        bits = rng.choice([4, 8])
        for max_rows in (0, most, 2 * most, 1):
            for max_kv in (0, max(h for h, _ in seqs), 1000):
                for p in forms(seqs, d, bits, heads, group, room, max_rows, max_kv, rows):
                    seen.add((p.tile, p.by_unit, p.share > 1, p.second > 0))
    for tile in (8, 16, 128) + ((256,) if d < 256 else ()):
        assert {(tile, True, False, False), (tile, False, True, True)} <= seen, (tile, seen)
