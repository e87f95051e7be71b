"""CPU checks of what libquant.h states of prefix_attention's workspace: what the
calls over either kind of tokens need, and every row's two results in fp32."""
import random

import bit_gemv_amd as bg


def test_the_workspace_is_both_calls_and_two_results_of_every_row():
    lib, rng = bg.load_library(), random.Random(4)
    for _ in range(300):
        heads, group, d, page = rng.choice([1, 2, 8]), rng.choice([1, 3, 8, 16]), rng.choice([64, 128, 256]), rng.choice([16, 64])
        b, p, rows = rng.choice([1, 4, 70]), rng.choice([0, 1, 3]), rng.choice([1, 5, 64, 700, 16384])
        qh, pages, front = heads * group, rng.choice([0, 3, 200]), rng.choice([0, 2, 300])
        hints = [rng.choice([0, 1, 40, rows]) for _ in range(2)] + [rng.choice([0, 500, 9000]) for _ in range(2)]
        own = lib.paged_attention_workspace_bytes(rows, qh, heads, d, b, pages, page, hints[0], hints[2])
        shared = lib.cross_attention_workspace_bytes(rows, qh, heads, d, p, front, page, hints[1], hints[3])
        need = lib.prefix_attention_workspace_bytes(rows, qh, heads, d, page, p, front, hints[1], hints[3], b, pages, hints[0],
                                                    hints[2])
        if p == 0:
            assert need == own
        else:
            assert 0 <= need - own - shared - 8 * rows * qh * (d + 2) < 1024


def test_sixteen_thousand_rows_of_64_heads():
    need = bg.load_library().prefix_attention_workspace_bytes(16384, 64, 8, 128, 64, 1, 32, 0, 0, 1, 256, 0, 0)
    assert 1.05e9 < need < 1.3e9
