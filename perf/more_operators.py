"""Measured cases of four operators over the quantized paged KV cache: attention
of a batch that shares long prefixes (each read once for all its rows), cross
attention to an encoder's states of another length, the attention weight that
every cached token has received, summed up call by call, and eviction from the
cache by that weight.

``run`` computes each operator in its plain form (elementary torch operations in
32 bits) or, with ``own``, by the calls a user makes of ``bit_gemv_amd``. What
the cache holds in codes is returned as the values they stand for. Head counts,
head sizes and token counts are those of the Llama-2-7B and -70B shaped
workloads, of one GPU's 8-way tensor-parallel share of the latter, and a small
64-wide head layout.
"""
import math
import random

import torch

own = False

PAGES_70B = dict(heads=8, group=8, dim=128, bits=8, sym=True, page=64)


def listed():
    return [
        # four requests of one system prompt on one of eight GPUs: the latency
        # of a decode step
        dict(name="prefix_decode_4", op="prefix", p=1, prefix=2011, b=4, rows=1, ctx=130, chunks=0, heads=1, group=8,
             dim=128, bits=8, sym=True, page=64),
        # a large decode batch behind one long prompt, 70B heads
        dict(name="prefix_decode_64", op="prefix", p=1, prefix=8192, b=64, rows=1, ctx=1024, chunks=0, **PAGES_70B),
        # ragged questions to three documents beside requests that already
        # decode, INT4 pages, 64-wide heads
        dict(name="prefix_chunks_3", op="prefix", p=3, prefix=6000, b=18, rows=200, ctx=900, chunks=12, heads=2, group=7,
             dim=64, bits=4, sym=False, page=16),
        # a decode batch of an encoder-decoder model, 7B heads: single tokens
        # over ragged encoder states
        dict(name="cross_decode_24", op="cross", b=24, rows=1, ctx=1500, chunks=0, heads=32, group=1, dim=128, bits=8,
             sym=False, page=32),
        # five beams of each of six inputs
        dict(name="cross_beams_6", op="cross", b=6, rows=5, ctx=3001, chunks=6, heads=8, group=2, dim=64, bits=4, sym=True,
             page=16),
        # a prompt of the decoder over a long input, 70B heads
        dict(name="cross_prompt_2", op="cross", b=2, rows=1100, ctx=8000, chunks=2, **PAGES_70B),
        # the weights of one decode step, one sequence on one of eight GPUs
        dict(name="weigh_decode_1", op="weigh", causal=True, b=1, rows=1, ctx=1003, chunks=0, heads=1, group=8, dim=128,
             bits=8, sym=True, page=64),
        # the weights of a large decode batch, long contexts, 70B heads
        dict(name="weigh_decode_64", op="weigh", causal=True, b=64, rows=1, ctx=16384, chunks=0, **PAGES_70B),
        # a prompt's last rows weigh the whole prompt, INT4 pages of the 7B stack
        dict(name="weigh_window_3", op="weigh", causal=True, b=3, rows=500, ctx=6000, chunks=3, heads=32, group=1, dim=128,
             bits=4, sym=False, page=16),
        # one sequence on one of eight GPUs back to half its pages
        dict(name="evict_1", op="evict", b=1, ctx=1003, keep=500, recent=64, heads=1, dim=128, bits=8, sym=True, page=64),
        # a batch back to a budget of 2048 tokens, 70B heads
        dict(name="evict_16", op="evict", b=16, ctx=8192, keep=2048, recent=256, heads=8, dim=128, bits=8, sym=True,
             page=64),
        # long ragged prompts of the 7B stack in INT4 after their prefill
        dict(name="evict_6_long", op="evict", b=6, ctx=30000, keep=4000, recent=1000, heads=32, dim=128, bits=4, sym=False,
             page=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefix", "cross", "weigh", "evict"])
    c = dict(op=op, dim=rng.choice([64, 128, 128, 256]), bits=rng.choice([4, 8]), sym=rng.choice([True, False]),
             page=rng.choice([16, 32, 64, 128]))
    if op == "evict":
        c.update(heads=rng.choice([1, 2, 5, 8, 32]), b=_log(rng, 1, 64))
        width = c["b"] * c["heads"] * c["dim"]
        c["ctx"] = _log(rng, 16, max(32, min(32768, 6 * 30000 * 32 * 128 // width)))
        c["keep"] = _log(rng, 1, max(1, min(c["ctx"], 6 * 2000 * 32 * 128 // width)))
        c["recent"] = rng.choice([0, rng.randint(0, c["keep"])])
        return c
    c.update(heads=rng.choice([1, 2, 5, 8]), group=rng.choice([1, 3, 7, 8, 16]))
    if op == "weigh":
        c["causal"] = rng.random() < 0.75
    width = c["heads"] * c["group"] * c["dim"]
    if rng.random() < 0.5:
        c.update(b=_log(rng, 1, 64), rows=1, chunks=0)
    else:
        c["b"] = _log(rng, 1, 12)
        c["chunks"] = rng.randint(1, c["b"])
        c["rows"] = _log(rng, 2, 600)
    seen = 2200 * 8000 * 64 * 128 // 2 // (max(1, c["chunks"]) * c["rows"] * width)   # keys a row may see
    held = 64 * 8000 * 8 * 128 // (c["b"] * c["heads"] * c["dim"])                   # and a sequence hold
    if op == "prefix":
        c["p"] = rng.choice([1, 1, 2, 3])
        c["ctx"] = c["rows"] + _log(rng, 1, max(2, min(2048, held, seen)))
        c["prefix"] = _log(rng, 16, max(32, min(16384, seen)))
    else:
        c["ctx"] = c["rows"] + _log(rng, 1, max(2, min(16384, held, seen)))
    return c


def _lengths(case):
    """(tokens held, rows) of each sequence: the first `chunks` have up to `rows`
    rows, the others one; a context is a quarter to all of `ctx`, the first one
    whole."""
    rng = random.Random("%d %d %d" % (case["b"], case["ctx"], case.get("rows", 0)))
    kv, new = [], []
    for i in range(case["b"]):
        n = 1
        if "rows" in case:
            n = case["rows"] if i == 0 else rng.randint(max(1, case["rows"] // 4), case["rows"]) if i < case["chunks"] else 1
        kv.append(max(n, case["ctx"] if i == 0 else rng.randint((case["ctx"] + 3) // 4, case["ctx"])))
        new.append(n)
    return kv, new


def _prefixes(case):
    """(tokens, sequences) of each shared prefix: consecutive sequences, about
    as many each; the first prefix has all its tokens, the others half or more."""
    rng = random.Random("%d %d" % (case["p"], case["prefix"]))
    cut = [case["b"] * j // case["p"] for j in range(case["p"] + 1)]
    return [(case["prefix"] if j == 0 else rng.randint((case["prefix"] + 1) // 2, case["prefix"]), cut[j + 1] - cut[j])
            for j in range(case["p"])]


def _mid(case):
    return 2 ** (case["bits"] - 1)


def _quantize(x, case):
    """Codes (unsigned), scale and zero of each last-axis vector, as the cache
    defines them."""
    if case["sym"]:
        qmax = _mid(case) - 1
        s = x.abs().amax(-1, keepdim=True).clamp_min(1e-8) / qmax
        return (torch.round(x / s).clamp(-qmax, qmax) + _mid(case)).to(torch.uint8), s, None
    top = 2 ** case["bits"] - 1
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = (hi - lo).clamp_min(1e-8) / top
    z = torch.round(-lo / s)
    return (torch.round(x / s) + z).clamp(0, top).to(torch.uint8), s, z


def _new_cache(case, pages, device):
    """An empty cache in the layout that include/libquant.h gives: keys
    [page][head][token][byte], values [page][head][token / 4][byte][token % 4]."""
    h, ps, row = case["heads"], case["page"], case["dim"] * case["bits"] // 8
    c = dict(k_codes=torch.zeros((pages, h, ps, row), dtype=torch.uint8, device=device),
             v_codes=torch.zeros((pages, h, ps // 4, row, 4), dtype=torch.uint8, device=device))
    for n in ("k_scales", "v_scales") + (() if case["sym"] else ("k_zeros", "v_zeros")):
        c[n] = torch.zeros((pages, h, ps), device=device)
    return c


def _fill(s, case, pages, normal):
    """Keys with a few large channels and even values in every slot of the pool,
    about a gigabyte at a time."""
    h, d, page, c = case["heads"], case["dim"], case["page"], s["cache"]
    loud = torch.where(normal(h, d) > 1.9, 4.0, 1.0)
    step = max(1, (1 << 28) // (h * d * page))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        for side in "kv":
            x = normal(n, h, page, d)
            q, scale, zero = _quantize(x * loud[:, None] if side == "k" else x, case)
            if case["bits"] == 4:
                q = q[..., 0::2] | (q[..., 1::2] << 4)
            if side == "v":
                q = q.view(n, h, page // 4, 4, -1).transpose(3, 4)
            c[side + "_codes"][a:a + n] = q
            c[side + "_scales"][a:a + n] = scale[..., 0]
            if zero is not None:
                c[side + "_zeros"][a:a + n] = zero[..., 0]


def _get(s, side, page, off, heads=slice(None)):
    """fp32 values [...][head][dim] of keys ("k") or values ("v") in the slots."""
    case, c = s["case"], s["cache"]
    q = c["k_codes"][:, heads][page, :, off] if side == "k" else c["v_codes"][:, heads][page, :, off // 4, :, off % 4]
    if case["bits"] == 4:
        q = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    z = _mid(case) if case["sym"] else c[side + "_zeros"][:, heads][page, :, off][..., None]
    return (q.float() - z) * c[side + "_scales"][:, heads][page, :, off][..., None]


def prepare(case, seed):
    device = torch.device("cuda")
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=device)

    def i32(values):
        return torch.tensor(values, dtype=torch.int32, device=device)

    s = dict(case=case)
    kv, new = _lengths(case)
    h, d, page, op = case["heads"], case["dim"], case["page"], case["op"]
    # every sequence's pages, those of the prefixes or of the evicted copies
    # behind them, scattered over the pool
    held = list(kv)
    if op == "prefix":
        held += [n for n, _ in _prefixes(case)]
    elif op == "evict":
        held += [min(n, case["keep"]) for n in kv]
    need = [(n + page - 1) // page for n in held]
    pages = sum(need) + 2
    order, at = torch.randperm(pages, generator=g, device=device).to(torch.int32).cpu(), 0
    tables = torch.full((len(held), max(need)), -1, dtype=torch.int32)
    for i, n in enumerate(need):
        tables[i, :n] = order[at:at + n]
        at += n
    b = case["b"]
    s["table"], s["kv"], s["max_kv"] = tables[:b, :max(need[:b])].to(device), i32(kv), max(kv)
    s["cache"] = _new_cache(case, pages, device)
    _fill(s, case, pages, normal)
    if op == "evict":
        # weights summed over many steps: a few tokens have most, many exactly none
        w = torch.exp(2 * normal(pages, h, page)) * (torch.rand((pages, h, page), generator=g, device=device) > 0.1)
        s["weights"] = w
        s["to"] = tables[b:, :max(need[b:])].to(device)
        ends = [0]
        for n in held[b:]:
            ends.append(ends[-1] + n)
        s["ends"], s["left"] = i32(ends), ends[-1]
        return s
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["starts"], s["rows"], s["max_rows"] = i32(starts), starts[-1], max(new)
    s["q"] = (normal(s["rows"], h * case["group"], d) * 1.5).to(torch.bfloat16)
    s["lse"] = torch.empty((s["rows"], h * case["group"]), device=device)
    if op == "prefix":
        parts = _prefixes(case)
        seqs = [0]
        for _, n in parts:
            seqs.append(seqs[-1] + n)
        s["prefix_table"] = tables[b:, :max(need[b:])].contiguous().to(device)
        s["prefix_kv"], s["prefix_starts"] = i32([n for n, _ in parts]), i32([starts[i] for i in seqs])
        s["max_prefix"] = max(n for n, _ in parts)
        s["max_prefix_rows"] = max(starts[j] - starts[i] for i, j in zip(seqs, seqs[1:]))
        s["host_prefix"] = [(n, starts[i], starts[j]) for (n, _), i, j in zip(parts, seqs, seqs[1:])]
    elif op == "weigh":
        # what the call's attention returned, and what earlier calls summed up
        s["lse"] = torch.cat([m + t.log() for m, t in _lse_parts(s)], 1).contiguous()
        s["weights"] = torch.exp(2 * normal(pages, h, page))
        s["out"] = torch.zeros_like(s["weights"])
    return s


def _rows_of(s):
    """(sequence, index in it, last position seen) of every row"""
    case = s["case"]
    row = torch.arange(s["rows"], device=s["kv"].device)
    seq = torch.searchsorted(s["starts"], row.to(torch.int32), right=True) - 1
    i = row - s["starts"][seq].long()
    held = s["kv"][seq].long()
    whole = case["op"] == "cross" or not case.get("causal", True)
    return seq, i, held - 1 if whole else held - (s["starts"][seq + 1] - s["starts"][seq]).long() + i


def _slots(s):
    """(page, offset) [b][max_kv] of every position, those past a sequence's end
    at its last one"""
    pos = torch.arange(s["max_kv"], device=s["kv"].device).expand(s["case"]["b"], -1)
    pos = torch.minimum(pos, s["kv"][:, None].long() - 1)
    return s["table"].long().gather(1, pos // s["case"]["page"]), pos % s["case"]["page"]


def _scores(s):
    """Per run of key heads: (heads, scale q . k fp32 [b][head][row][group][key],
    -inf where a row does not see the key)"""
    case = s["case"]
    h, g, d, b = case["heads"], case["group"], case["dim"], case["b"]
    seq, i, last = _rows_of(s)
    page, off = _slots(s)
    end = torch.full((b, s["max_rows"]), -1, device=page.device)
    end[seq, i] = last
    unseen = torch.arange(s["max_kv"], device=page.device) > end[:, :, None]
    step = max(1, (1 << 29) // (b * s["max_kv"] * (d + g * s["max_rows"])))
    for h0 in range(0, h, step):
        part = slice(h0, min(h, h0 + step))
        n = part.stop - h0
        q = torch.zeros((b, s["max_rows"], n, g, d), device=page.device)
        q[seq, i] = s["q"].float().view(-1, h, g, d)[:, part]
        q = q.permute(0, 2, 1, 3, 4).reshape(b, n, -1, d)
        k = _get(s, "k", page, off, part).permute(0, 2, 3, 1).contiguous()
        t = (q @ k).mul_(d ** -0.5).view(b, n, s["max_rows"], g, -1)
        yield part, t.masked_fill_(unseen[:, None, :, None, :], -math.inf)


def _lse_parts(s):
    """Per run of key heads: maximum and sum of the rows' scores [rows][q heads]"""
    seq, i, _ = _rows_of(s)
    for _, t in _scores(s):
        m = t.amax(-1)
        total = t.sub_(m.clamp_min(-3e38)[..., None]).exp_().sum(-1)
        yield tuple(x.permute(0, 2, 1, 3)[seq, i].flatten(1) for x in (m, total))


def _own_part(s):
    """Maximum, sum and weighted values of the rows over their sequences' tokens:
    [rows][q heads] twice and [rows][q heads][dim]"""
    case = s["case"]
    seq, i, _ = _rows_of(s)
    page, off = _slots(s)
    parts = []
    for heads, t in _scores(s):
        v = _get(s, "v", page, off, heads).transpose(1, 2).contiguous()
        m = t.amax(-1).clamp_min(-3e38)
        t.sub_(m[..., None]).exp_()
        o = (t.flatten(2, 3) @ v).view(*t.shape[:4], case["dim"])
        parts.append([x.transpose(1, 2)[seq, i].flatten(1, 2) for x in (m, t.sum(-1), o)])
    return [torch.cat(x, 1) for x in zip(*parts)]


def _plain_prefix(s):
    case = s["case"]
    h, g, d = case["heads"], case["group"], case["dim"]
    m, total, o = _own_part(s)
    outs, sums = [], []
    for j, (n, a, z) in enumerate(s["host_prefix"]):
        pos = torch.arange(n, device=m.device)
        page, off = s["prefix_table"][j, pos // case["page"]].long(), pos % case["page"]
        k = _get(s, "k", page, off).permute(1, 2, 0).contiguous()
        v = _get(s, "v", page, off).transpose(0, 1).contiguous()
        q = s["q"][a:z].float().view(-1, h, g, d).transpose(0, 1).reshape(h, -1, d)
        t = (q @ k).mul_(d ** -0.5)
        top = t.amax(-1, keepdim=True)
        t.sub_(top).exp_()

        def rows(x):
            return x.view(h, -1, g, x.shape[-1]).transpose(0, 1).flatten(1, 2)

        pm, pt, po = rows(top)[..., 0], rows(t.sum(-1, keepdim=True))[..., 0], rows(t @ v)
        both = torch.maximum(pm, m[a:z])
        x, y = torch.exp(pm - both), torch.exp(m[a:z] - both)
        pt = pt * x + total[a:z] * y
        outs.append((po * x[..., None] + o[a:z] * y[..., None]) / pt[..., None])
        sums.append(both + pt.log())
    return {"out": torch.cat(outs).to(torch.bfloat16), "lse": torch.cat(sums)}


def _plain_cross(s):
    m, total, o = _own_part(s)
    return {"out": (o / total.clamp_min(1e-30)[..., None]).to(torch.bfloat16), "lse": m + total.log()}


def _plain_weigh(s):
    case = s["case"]
    seq, i, _ = _rows_of(s)
    page, off = _slots(s)
    b, g, h = case["b"], case["group"], case["heads"]
    lse = torch.zeros((b, s["max_rows"], h, g), device=page.device)
    lse[seq, i] = s["lse"].view(-1, h, g)
    pos = torch.arange(s["max_kv"], device=page.device)
    held = pos < s["kv"][:, None]
    # a token that the call's rows brought has no weight from before
    old = pos < (s["kv"] - (s["starts"][1:] - s["starts"][:-1]) if case["causal"] else s["kv"])[:, None]
    at, slot = (page[held], off[held]), held.nonzero(as_tuple=True)
    for heads, t in _scores(s):
        w = t.sub_(lse[:, :, heads].transpose(1, 2)[..., None]).exp_().sum((2, 3)).transpose(1, 2)
        w = w[slot] + s["weights"][:, heads][at[0], :, at[1]] * old[slot][:, None]
        s["out"][:, heads][at[0], :, at[1]] = w
    return {"weights": s["out"]}


def _plain_evict(s):
    case, c = s["case"], s["cache"]
    b, h, keep, recent = case["b"], case["heads"], case["keep"], case["recent"]
    page, off = _slots(s)
    n = s["kv"].long()[:, None]
    pos = torch.arange(s["max_kv"], device=page.device)
    w = s["weights"][page, :, off].transpose(1, 2)                          # [b][head][key]
    w = torch.where((pos >= n - recent)[:, None], math.inf, w).masked_fill((pos >= n)[:, None], -1.0)
    best = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    left = n.clamp_max(keep)
    late = (torch.arange(best.shape[-1], device=page.device) >= left)[:, None]
    best = best.masked_fill(late, 1 << 30).sort(-1).values
    kept = torch.full((b, h, keep), -1, dtype=torch.int32, device=page.device)
    kept[..., :best.shape[-1]] = torch.where(late, -1, best)
    seq, head, j = (kept >= 0).nonzero(as_tuple=True)
    src = kept[seq, head, j].long()
    p0, o0, p1, o1 = page[seq, src], off[seq, src], s["to"][seq, j // case["page"]].long(), j % case["page"]
    for name in ("k_codes", "k_scales", "v_scales", "k_zeros", "v_zeros"):
        if name in c:
            c[name][p1, head, o1] = c[name][p0, head, o0]
    c["v_codes"][p1, head, o1 // 4, :, o1 % 4] = c["v_codes"][p0, head, o0 // 4, :, o0 % 4]
    s["weights"][p1, head, o1] = s["weights"][p0, head, o0]
    pos = torch.arange(s["to"].shape[1] * case["page"], device=page.device)
    seq, j = (pos < left).nonzero(as_tuple=True)
    at = s["to"][seq, j // case["page"]].long(), j % case["page"]
    return {"lens": left[:, 0].to(torch.int32), "kept": kept, "weights": s["weights"],
            "k": _get(s, "k", *at).to(torch.bfloat16), "v": _get(s, "v", *at).to(torch.bfloat16)}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"prefix": _plain_prefix, "cross": _plain_cross, "weigh": _plain_weigh, "evict": _plain_evict}[op](s)
    import bit_gemv_amd as bg
    c = s["cache"]
    cache = bg.KVCache(c["k_codes"], c["v_codes"], c["k_scales"], c["v_scales"], c.get("k_zeros"), c.get("v_zeros"),
                       case["dim"], case["bits"])
    if op == "evict":
        # into other pages, so that a pass finds the batch as the last one did
        lens, kept = bg.kv_cache_evict(cache, s["weights"], s["table"], s["kv"], case["keep"], case["recent"],
                                       to_table=s["to"], max_kv=s["max_kv"])
        k, v = bg.kv_cache_read(cache, s["to"], lens, s["ends"], rows=s["left"])
        return {"lens": lens, "kept": kept, "weights": s["weights"], "k": k, "v": v}
    batch, bounds = (s["table"], s["kv"], s["starts"]), dict(max_rows=s["max_rows"], max_kv=s["max_kv"])
    if op == "weigh":
        return {"weights": bg.kv_cache_weigh(s["q"], s["lse"], cache, s["weights"], *batch, causal=case["causal"],
                                             out=s["out"], **bounds)}
    if op == "cross":
        return {"out": bg.cross_attention(s["q"], cache, *batch, lse=s["lse"], **bounds), "lse": s["lse"]}
    out = bg.prefix_attention(s["q"], cache, s["prefix_table"], s["prefix_kv"], s["prefix_starts"], *batch, lse=s["lse"],
                              max_prefix_rows=s["max_prefix_rows"], max_prefix=s["max_prefix"], **bounds)
    return {"out": out, "lse": s["lse"]}


def work(case):
    kv, new = _lengths(case)
    h, d = case["heads"], case["dim"]
    half = h * (d * case["bits"] // 8 + (4 if case["sym"] else 8))         # one token's keys, or its values
    if case["op"] == "evict":
        # the weights, the tokens that stay in and out, and their values out
        left = sum(min(n, case["keep"]) for n in kv)
        return {"bytes": sum(kv) * h * 4 + left * (2 * 2 * half + 2 * h * d * 2 + h * 8) + left * 2 * half,
                "flops": sum(kv) * h + left * 4 * h * d}
    heads, rows = h * case["group"], sum(new)
    pairs = list(zip(kv, new))
    seen = sum(m * n for m, n in pairs)
    if case["op"] == "prefix" or case.get("causal", False):
        seen = sum(n * (m - n) + n * (n + 1) // 2 for m, n in pairs)
    if case["op"] == "weigh":
        return {"bytes": sum(kv) * (half + 2 * h * 4) + rows * heads * (d * 2 + 4), "flops": 2 * d * heads * seen}
    tokens = sum(kv)  # of attention: q in, the rows and their log-sum-exp out
    if case["op"] == "prefix":
        at = 0
        for n, seqs in _prefixes(case):
            tokens += n
            seen += n * sum(new[at:at + seqs])
            at += seqs
    return {"bytes": tokens * 2 * half + rows * heads * (d * 4 + 4), "flops": 4 * d * heads * seen}


def _wide(s, pages, head, side):
    """64-bit values [token][dim] of one head in a list of pages"""
    case, c = s["case"], s["cache"]
    code = c[side + "_codes"][pages, head]
    if side == "v":
        code = code.transpose(2, 3).flatten(1, 2)
    code = code.reshape(-1, code.shape[-1])
    full = torch.empty((code.shape[0], case["dim"]), dtype=torch.float64, device=code.device)
    if case["bits"] == 8:
        full.copy_(code)
    else:
        full[:, 0::2], full[:, 1::2] = code % 16, code // 16
    zero = _mid(case) if case["sym"] else c[side + "_zeros"][pages, head].double().view(-1, 1)
    return (full - zero) * c[side + "_scales"][pages, head].double().view(-1, 1)


def exact(case, seed):
    s = prepare(case, seed)
    kv, new = _lengths(case)
    h, g, d, page, op = case["heads"], case.get("group", 1), case["dim"], case["page"], case["op"]
    device, f8 = s["kv"].device, torch.float64
    lists = [s["table"][i, :(m + page - 1) // page].long() for i, m in enumerate(kv)]
    if op == "evict":
        after, values, all_kept = s["weights"].double(), {"k": [], "v": []}, torch.full(
            (case["b"], h, case["keep"]), -1, dtype=torch.int32, device=device)
        for i, m in enumerate(kv):
            n, sides = min(m, case["keep"]), {"k": [], "v": []}
            for j in range(h):
                w = s["weights"][lists[i], j].view(-1)[:m]
                old = max(0, m - min(case["recent"], n))
                # the largest of the older ones, the earlier of equals, then the recent ones
                top = torch.argsort(-w[:old], stable=True)[:n - (m - old)].sort().values
                stay = torch.cat((top, torch.arange(old, m, device=device)))
                all_kept[i, j, :n] = stay.to(torch.int32)
                to, at = s["to"][i].long(), torch.arange(n, device=device)
                after[to[at // page], j, at % page] = w[stay].double()
                for side in "kv":
                    sides[side].append(_wide(s, lists[i], j, side)[stay])
            for side in "kv":
                values[side].append(torch.stack(sides[side], 1))
        lens = torch.tensor([min(m, case["keep"]) for m in kv], dtype=torch.int32, device=device)
        return {"lens": lens, "kept": all_kept, "weights": after, "k": torch.cat(values["k"]), "v": torch.cat(values["v"])}
    out, lse = torch.empty(s["q"].shape, dtype=f8, device=device), s["lse"].double()
    sums = None if op != "weigh" else s["out"].double()
    prefix_of = [j for j, (_, n) in enumerate(_prefixes(case)) for _ in range(n)] if op == "prefix" else None
    at = 0
    for i, (m, n) in enumerate(zip(kv, new)):
        first = m - n if op == "prefix" or case.get("causal", False) else m
        late = torch.arange(m, device=device)[None, :] > torch.arange(first, first + n, device=device)[:, None]
        for j in range(h):
            k = _wide(s, lists[i], j, "k")[:m]
            front = 0
            if op == "prefix":
                front = s["host_prefix"][prefix_of[i]][0]
                shared = s["prefix_table"][prefix_of[i], :(front + page - 1) // page].long()
                k = torch.cat((_wide(s, shared, j, "k")[:front], k))
            if op != "weigh":
                v = _wide(s, lists[i], j, "v")[:m]
                v = v if op == "cross" else torch.cat((_wide(s, shared, j, "v")[:front], v))
            total = torch.zeros(m, dtype=f8, device=device)
            for x in range(j * g, (j + 1) * g):
                logit = s["q"][at:at + n, x].to(f8) @ k.T / math.sqrt(d)
                logit[:, front:].masked_fill_(late, -math.inf)
                if op == "weigh":
                    total += torch.exp(logit - s["lse"][at:at + n, x].to(f8)[:, None]).sum(0)
                else:
                    out[at:at + n, x] = torch.softmax(logit, -1) @ v
                    lse[at:at + n, x] = torch.logsumexp(logit, -1)
            if op == "weigh":
                where = lists[i].repeat_interleave(page)[:m], torch.arange(m, device=device) % page
                before = s["weights"][where[0], j, where[1]].double()
                before[min(first, m):] = 0
                sums[where[0], j, where[1]] = total + before
        at += n
    return {"out": out, "lse": lse} if op != "weigh" else {"weights": sums}
