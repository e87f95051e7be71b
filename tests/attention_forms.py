"""The forms that paged_attention's work takes, worked out on the host from the
rules that the library states, so that a test can say which of them it reaches:
tiles of 8, 16, 128 or 256 rows, whole units or spans, parts and their join.
The model is held to the library by the workspace it predicts."""
import bit_gemv_amd as bg

FEW_STEP = 128


class Pass:
    """One launch: rows of a tile, keys of a step, blocks a key head, and what
    its units are cut into. Steps of all units lie one after another; block i
    takes steps [i share, (i + 1) share)."""

    def __init__(self, tile, step, cap, by_unit, least, most, seqs, group, room):
        self.tile, self.step, self.by_unit = tile, step, by_unit
        self.units = []
        for held, n in seqs:
            if n and least <= n * group <= most:
                keys = max(1, min(held, room))
                steps = 1 if by_unit else -(-keys // step)
                self.units += [steps] * -(-n * group // tile)
        self.share = max(1, -(-sum(self.units) // cap))
        self.cap = cap
        at, self.parts, self.second, self.longest, self.keys_in_a_piece = 0, [], 0, 0, 0
        for steps in self.units:
            cuts = [c for c in range(at - at % self.share, at + steps + self.share, self.share) if at < c < at + steps]
            ends = [at] + cuts + [at + steps]
            pieces = [b - a for a, b in zip(ends, ends[1:])]
            self.longest = max([self.longest] + pieces)
            if cuts:
                self.parts.append(pieces)
                # a part that is not its block's first piece takes the block's second place
                self.second += at % self.share != 0
            at += steps

    def __repr__(self):
        return (f"tile {self.tile} {'units' if self.by_unit else 'spans'} {len(self.units)} of {sum(self.units)} steps, cap "
                f"{self.cap}, share {self.share}, cut {len(self.parts)}, second places {self.second}, longest piece {self.longest}")


def forms(seqs, d, bits, heads, group, room, max_rows, max_kv, rows):
    """The launches of a call with these hints over `rows` rows, the workspace
    they need checked against the library's."""
    b = len(seqs)
    n = rows if max_rows <= 0 or max_rows > rows else max_rows
    kv = room if max_kv <= 0 or max_kv > room else max_kv
    ceil = lambda x, y: -(-x // y)  # noqa: E731

    def one(tile, rows, n, least, most):
        units, tiles = ceil(rows * group, tile) + b, ceil(n * group, tile)
        step = FEW_STEP if tile < 128 else tile // (2 if d == 64 else 4)
        unit_steps, likely = max(1, ceil(kv, step)), min(b * tiles, units)
        blocks = lambda bits: 256 if tile == 256 else 768 if tile == 8 and d <= 128 and d * bits <= 512 else 512  # noqa: E731
        if tile >= 128:
            slots, load = (256 if tile == 256 or d == 256 else 512), likely * heads
            mean = kv - min(n, kv) // 2 if b == 1 else kv // 2
            prior, idle = max(0, kv - n), ceil(load, slots) * slots - load
            by_unit = load >= 4 * slots or (kv <= load * mean // slots + 1200
                                            and (idle * prior <= 1200 * slots if b == 1 else prior <= 1200))
        else:
            by_unit = kv <= 1024 or (kv <= 2048 and likely * heads >= 256)
        cap, most_cap = (min(likely if by_unit else ceil(blocks(x), heads), units * unit_steps) for x in (bits, 4))
        need = 2 * most_cap * heads * tile * (d + 2) * 4 if most_cap > 1 and not by_unit else 0
        return Pass(tile, step, cap, by_unit, least, most, seqs, group, room), ceil(need, 256) * 256

    if n * group <= 16:
        launches = [one(8 if n * group <= 8 else 16, rows, n, 1, 1 << 40)]
    else:
        tile = 256 if rows * group >= 256 * b and d != 256 else 128
        mixed = b >= 4 and group <= 16 and (rows - n) * group <= 64 * (b - 1)
        launches = [one(tile, rows, n, 17 if mixed else 1, 1 << 40)]
        if mixed:
            launches.append(one(16, 0, 1, 1, 16))
    need = sum(x[1] for x in launches)
    page = 16 if room % 16 == 0 else 1
    got = bg.load_library().paged_attention_workspace_bytes(rows, heads * group, heads, d, b, room // page, page, max_rows,
                                                            max_kv)
    assert got == need, (got, need, [x[0] for x in launches])
    return [x[0] for x in launches]
