"""Measured cases of the serving operators: the residual norm into INT8, the
quantized paged KV cache (written and read back) and attention over it.

``run`` computes each operator in its plain form (elementary torch
operations in 32 bits, the norm's sum of squares in 64) or, with ``own``, by
the calls a user makes of ``bit_gemv_amd``. Codes are returned as the values
they stand for. Head counts, head sizes, hidden sizes and token counts are
those of the Llama-2-7B and -70B shaped workloads, of one GPU's 8-way
tensor-parallel share of the latter, and a small 64-wide head layout.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one decode step of the 70B stack: the attention block's fp32 product
        # joins the residual and becomes the next W8A8 product's INT8 input
        dict(name="norm_decode_1", op="norm", t=1, k=8192, x="fp32", res="bf16", w="bf16"),
        # a ragged prefill of the 7B stack; the norm weight has the smoothing
        # factors folded in, so it is fp32
        dict(name="norm_prefill_509", op="norm", t=509, k=4096, x="bf16", res="bf16", w="fp32"),
        # a large prefill batch of the 70B stack
        dict(name="norm_prefill_8192", op="norm", t=8192, k=8192, x="fp32", res="bf16", w="bf16"),
        # a decode batch appends one token per sequence, 70B heads
        dict(name="cache_append_16", op="cache", b=16, rows=1, ctx=4096, chunks=0, heads=8, dim=128, bits=8,
             sym=True, page=64, x="bf16"),
        # ragged prompts of the 7B stack into INT4 pages, straight from the
        # fp32 products
        dict(name="cache_chunks_5", op="cache", b=5, rows=512, ctx=1500, chunks=5, heads=32, dim=128, bits=4,
             sym=False, page=16, x="fp32"),
        # long prompts of the 70B stack
        dict(name="cache_prefill_4", op="cache", b=4, rows=8192, ctx=8192, chunks=4, heads=8, dim=128, bits=8,
             sym=True, page=64, x="bf16"),
        # one sequence on one of eight GPUs: the latency of a decode step
        dict(name="attn_decode_1", op="attn", b=1, rows=1, ctx=1003, chunks=0, heads=1, group=8, dim=128, bits=8,
             sym=True, page=64),
        # an ordinary decode batch over INT4 pages, 70B heads
        dict(name="attn_decode_16", op="attn", b=16, rows=1, ctx=8192, chunks=0, heads=8, group=8, dim=128, bits=4,
             sym=False, page=32),
        # a large decode batch, long contexts, 70B heads
        dict(name="attn_decode_64", op="attn", b=64, rows=1, ctx=16384, chunks=0, heads=8, group=8, dim=128, bits=8,
             sym=True, page=64),
        # a 2048-token chunk over an 8192-token context, 70B heads
        dict(name="attn_chunk_2048", op="attn", b=1, rows=2048, ctx=8192, chunks=1, heads=8, group=8, dim=128, bits=8,
             sym=True, page=64),
        # two prompt chunks scheduled beside ten decoding sequences, 7B heads
        dict(name="attn_mixed_12", op="attn", b=12, rows=700, ctx=4001, chunks=2, heads=32, group=1, dim=128, bits=4,
             sym=True, page=16),
        # ragged chunks with 64-wide heads
        dict(name="attn_chunks_d64", op="attn", b=4, rows=1000, ctx=4096, chunks=4, heads=2, group=7, dim=64, bits=8,
             sym=False, page=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "cache", "attn"])
    if op == "norm":
        k = 128 * _log(rng, 8, 224)
        t = _log(rng, 1, max(1, (8192 * 8192) // k))
        return dict(op="norm", t=t, k=k, x=rng.choice(["bf16", "fp32"]), res=rng.choice(["bf16", "bf16", "fp32", "none"]),
                    w=rng.choice(["bf16", "fp32"]))
    c = dict(op=op, dim=rng.choice([64, 128, 128, 256]), bits=rng.choice([4, 8]), sym=rng.choice([True, False]),
             page=rng.choice([16, 32, 64, 128]))
    if op == "cache":
        c.update(heads=rng.choice([1, 2, 5, 8, 32]), x=rng.choice(["bf16", "fp32"]))
        most = 32768 * 8 * 128 // (c["heads"] * c["dim"])
        c["b"] = _log(rng, 1, 64)
        c["rows"] = _log(rng, 1, min(4096, max(1, most // c["b"])))
        c["chunks"] = c["b"] if c["rows"] > 1 else 0
        c["ctx"] = c["rows"] + rng.randrange(0, 4096)
        return c
    c.update(heads=rng.choice([1, 2, 5, 8]), group=rng.choice([1, 3, 7, 8, 16]))
    if rng.random() < 0.5:
        c.update(b=_log(rng, 1, 64), rows=1, chunks=0)
        most = 64 * 8192 * 8 * 128 // (c["b"] * c["heads"] * c["dim"])
        c["ctx"] = _log(rng, 1, max(2, min(16384, most)))
    else:
        c["b"] = _log(rng, 1, 8)
        c["chunks"] = rng.randrange(1, c["b"] + 1)
        c["rows"] = _log(rng, 2, 1024)
        most = 2048 * 8192 * 64 * 128 // (2 * c["b"] * c["rows"] * c["heads"] * c["group"] * c["dim"])
        c["ctx"] = c["rows"] + _log(rng, 1, max(2, min(8192, most)))
    return c


def _lengths(case):
    """(tokens held, new tokens) of each sequence: the first `chunks` bring up
    to `rows` new tokens, the others one; a context is a quarter to all of
    `ctx`, the first one whole."""
    rng = random.Random("%(b)d %(rows)d %(ctx)d %(chunks)d" % case)
    kv, new = [], []
    for i in range(case["b"]):
        n = case["rows"] if i == 0 else rng.randint(max(1, case["rows"] // 4), case["rows"]) if i < case["chunks"] else 1
        kv.append(max(n, case["ctx"] if i == 0 else rng.randint((case["ctx"] + 3) // 4, case["ctx"])))
        new.append(n)
    return kv, new


def _levels(bits, sym):
    """(largest code, the code that stands for zero where it is fixed)"""
    return (2 ** bits - 1, 2 ** (bits - 1) if sym else 0)


def _quantize(x, bits, sym):
    """Codes (unsigned), scale and zero of each last-axis vector, as
    quantize_groupwise defines them with one group per vector."""
    top, mid = _levels(bits, sym)
    if sym:
        qmax = 2 ** (bits - 1) - 1
        s = x.abs().amax(-1, keepdim=True).clamp_min(1e-8) / qmax
        return (torch.round(x / s).clamp(-qmax, qmax) + mid).to(torch.uint8), s, None
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = (hi - lo).clamp_min(1e-8) / top
    z = torch.round(-lo / s)
    return (torch.round(x / s) + z).clamp(0, top).to(torch.uint8), s, z


def _nibbles(codes, bits):
    """[..., dim] codes to bytes: as they are, or two neighbours in one byte"""
    return codes if bits == 8 else codes[..., 0::2] | (codes[..., 1::2] << 4)


def _codes(b, bits):
    return b if bits == 8 else torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _new_cache(case, pages, device):
    """An empty cache in the layout that include/libquant.h gives: keys
    [page][head][token][byte], values [page][head][token / 4][byte][token % 4]."""
    h, ps, db = case["heads"], case["page"], case["dim"] * case["bits"] // 8
    c = dict(k_codes=torch.zeros((pages, h, ps, db), dtype=torch.uint8, device=device),
             v_codes=torch.zeros((pages, h, ps // 4, db, 4), dtype=torch.uint8, device=device))
    for n in ("k_scales", "v_scales") + (() if case["sym"] else ("k_zeros", "v_zeros")):
        c[n] = torch.zeros((pages, h, ps), device=device)
    return c


def _put(c, case, at, k, v):
    """Quantize k, v [rows][head][dim] into the slots `at` = (page, offset)."""
    page, off = at
    for n, x in (("k", k), ("v", v)):
        q, s, z = _quantize(x, case["bits"], case["sym"])
        q = _nibbles(q, case["bits"])
        if n == "k":
            c["k_codes"][page, :, off] = q
        else:
            c["v_codes"][page, :, off // 4, :, off % 4] = q
        c[n + "_scales"][page, :, off] = s[..., 0]
        if z is not None:
            c[n + "_zeros"][page, :, off] = z[..., 0]


def _get(c, case, at, n, dtype=torch.float32):
    """The values [rows][head][dim] of keys ("k") or values ("v") in the slots."""
    page, off = at
    q = c["k_codes"][page, :, off] if n == "k" else c["v_codes"][page, :, off // 4, :, off % 4]
    q = _codes(q, case["bits"]).to(dtype)
    z = _levels(case["bits"], True)[1] if case["sym"] else c[n + "_zeros"][page, :, off][..., None].to(dtype)
    return (q - z) * c[n + "_scales"][page, :, off][..., None].to(dtype)


def _slots(case, table, seq, pos):
    return table[seq, pos // case["page"]].long(), pos % case["page"]


def prepare(case, seed):
    device = torch.device("cuda")
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=device)

    s = dict(case=case)
    if case["op"] == "norm":
        t, k = case["t"], case["k"]
        # a few channels carry outliers, as activations do
        out = torch.where(torch.rand(k, generator=g, device=device) < 0.002, 20.0, 1.0)
        s["x"] = (normal(t, k) * out).to(TYPES[case["x"]])
        s["res"] = None if case["res"] == "none" else (normal(t, k) * out * 2).to(TYPES[case["res"]])
        s["w"] = (1 + 0.1 * normal(k)).to(TYPES[case["w"]])
        s["values"] = torch.empty((t, k), dtype=torch.bfloat16, device=device)
        return s
    kv, new = _lengths(case)
    page = case["page"]
    need = [(n + page - 1) // page for n in kv]
    pages, wide = sum(need) + 2, max(need)
    order = torch.randperm(pages, generator=g, device=device).to(torch.int32)
    table = torch.full((len(kv), wide), -1, dtype=torch.int32)
    order, at = order.cpu(), 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["table"] = table.to(device)
    s["kv"] = torch.tensor(kv, dtype=torch.int32, device=device)
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device=device)
    s["rows"], s["max_rows"], s["max_kv"] = starts[-1], max(new), max(kv)
    s["cache"] = c = _new_cache(case, pages, device)
    h, d = case["heads"], case["dim"]
    # keys have a few large channels, values are even
    key = torch.where(torch.rand(h, d, generator=g, device=device) < 0.03, 4.0, 1.0)
    if case["op"] == "attn":
        # every page of the pool is filled, page by page of about a gigabyte
        slots = torch.arange(pages * page, device=device)
        step = max(page, (1 << 28) // (h * d))
        for a in range(0, pages * page, step):
            part = slots[a:a + step]
            _put(c, case, (part // page, part % page), normal(len(part), h, d) * key, normal(len(part), h, d))
        s["q"] = (normal(s["rows"], h * case["group"], d) * 1.5).to(torch.bfloat16)
    else:
        s["k"] = (normal(s["rows"], h, d) * key).to(TYPES[case["x"]])
        s["v"] = normal(s["rows"], h, d).to(TYPES[case["x"]])
    return s


def _plain_norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    r = torch.rsqrt((h.double() * h.double()).mean(-1, keepdim=True) + EPS).float()
    y = (h * r) * s["w"].float()
    sx = y.abs().amax(-1, keepdim=True).clamp_min(1e-8) / 127
    q = torch.round(y / sx).clamp(-127, 127)
    return {"values": (q * sx).to(torch.bfloat16), "sx": sx[:, 0],
            "residual": None if s["res"] is None else h.to(s["res"].dtype)}


def _new_rows(s):
    """(sequence, position) of every new token"""
    row = torch.arange(s["rows"], device=s["kv"].device)
    seq = torch.searchsorted(s["starts"], row.to(torch.int32), right=True) - 1
    return seq, s["kv"][seq].long() - s["starts"][seq + 1].long() + row


def _plain_cache(s):
    case, c = s["case"], s["cache"]
    at = _slots(case, s["table"], *_new_rows(s))
    _put(c, case, at, s["k"].float(), s["v"].float())
    return {"k": _get(c, case, at, "k").to(torch.bfloat16), "v": _get(c, case, at, "v").to(torch.bfloat16)}


def _plain_attn(s):
    case, c = s["case"], s["cache"]
    b, h, g, d = case["b"], case["heads"], case["group"], case["dim"]
    pos = torch.arange(s["max_kv"], device=s["kv"].device).expand(b, -1)
    seq = torch.arange(b, device=s["kv"].device)[:, None].expand_as(pos)
    at = _slots(case, s["table"], seq, torch.minimum(pos, s["kv"][:, None].long() - 1))
    k = _get(c, case, at, "k").transpose(1, 2)                        # [b][head][key][dim]
    v = _get(c, case, at, "v").transpose(1, 2)
    row_seq, row_pos = _new_rows(s)
    i = torch.arange(s["rows"], device=s["kv"].device) - s["starts"][row_seq].long()
    q = torch.zeros((b, s["max_rows"], h, g, d), device=k.device)
    q[row_seq, i] = s["q"].float().view(-1, h, g, d)
    last = torch.full((b, s["max_rows"]), -1, device=k.device)
    last[row_seq, i] = row_pos
    q = q.permute(0, 2, 1, 3, 4).reshape(b, h, -1, d)                  # rows of one key head together
    p = (q @ k.transpose(2, 3).contiguous()).mul_(d ** -0.5).view(b, h, -1, g, s["max_kv"])
    p.masked_fill_(pos[:, None, None, None, :] > last[:, None, :, None, None], -math.inf)
    m = p.amax(-1, keepdim=True).clamp_min(-3e38)
    p.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).view(b, h, -1, g, d) / total.clamp_min(1e-30)
    o = o.permute(0, 2, 1, 3, 4)[row_seq, i].reshape(-1, h * g, d)
    return {"out": o.to(torch.bfloat16)}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "cache": _plain_cache, "attn": _plain_attn}[op](s)
    import bit_gemv_amd as bg
    if op == "norm":
        qx, sx, res = bg.rms_norm_int8(s["x"], s["w"], eps=EPS, residual=s["res"])
        return {"values": torch.mul(qx, sx[:, None], out=s["values"]), "sx": sx, "residual": res}
    c, batch = s["cache"], (s["table"], s["kv"], s["starts"])
    cache = bg.KVCache(c["k_codes"], c["v_codes"], c["k_scales"], c["v_scales"], c.get("k_zeros"), c.get("v_zeros"),
                       s["case"]["dim"], s["case"]["bits"])
    if op == "cache":
        bg.kv_cache_write(s["k"], s["v"], cache, *batch, max_rows=s["max_rows"])
        k, v = bg.kv_cache_read(cache, *batch, rows=s["rows"], max_rows=s["max_rows"])
        return {"k": k, "v": v}
    return {"out": bg.paged_attention(s["q"], cache, *batch, max_rows=s["max_rows"], max_kv=s["max_kv"])}


def work(case):
    size = {"bf16": 2, "fp32": 4, "none": 0}
    if case["op"] == "norm":
        n = case["t"] * case["k"]
        return {"bytes": n * (size[case["x"]] + 2 * size[case["res"]] + 1) + case["k"] * size[case["w"]] + 4 * case["t"],
                "flops": 8 * n}
    kv, new = _lengths(case)
    h, d = case["heads"], case["dim"]
    token = 2 * h * (d * case["bits"] // 8 + (4 if case["sym"] else 8))   # one token's keys and values
    if case["op"] == "cache":
        # the new keys and values in, their codes out and in again, the values out
        n = sum(new)
        return {"bytes": n * (2 * h * d * (size[case["x"]] + 2) + 2 * token), "flops": 8 * n * 2 * h * d}
    heads = h * case["group"]
    seen = sum(n * (m - n) + n * (n + 1) // 2 for m, n in zip(kv, new))
    return {"bytes": sum(kv) * token + sum(new) * heads * d * 4, "flops": 4 * d * heads * seen}


def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "norm":
        h = s["x"].to(f8) + (0 if s["res"] is None else s["res"].to(f8))
        y = h / (h.square().sum(-1, keepdim=True) / case["k"] + EPS).sqrt() * s["w"].to(f8)
        sx = y.abs().amax(-1).clamp_min(1e-8) / 127
        q = (y / sx[:, None]).round().clamp(-127, 127)
        return {"values": q * sx[:, None], "sx": sx, "residual": None if s["res"] is None else h}
    kv, new = _lengths(case)
    if case["op"] == "cache":
        outs = {}
        top = 2 ** case["bits"] - 1
        for n in ("k", "v"):
            x = s[n].to(f8)
            if case["sym"]:
                step = x.abs().amax(-1, keepdim=True).clamp_min(1e-8) / (top // 2)
                outs[n] = (x / step).round() * step
            else:
                lo = x.amin(-1, keepdim=True)
                step = (x.amax(-1, keepdim=True) - lo).clamp_min(1e-8) / top
                z = (-lo / step).round()
                outs[n] = (((x / step).round() + z).clamp(0, top) - z) * step
        return outs
    out, at = torch.empty(s["q"].shape, dtype=f8, device=s["q"].device), 0
    g, d, page = case["group"], case["dim"], case["page"]
    for i, (m, n) in enumerate(zip(kv, new)):
        pages = s["table"][i, :(m + page - 1) // page].long()
        late = torch.arange(m, device=out.device)[None, :] > torch.arange(m - n, m, device=out.device)[:, None]
        for h in range(case["heads"]):
            side = []
            for name in ("k", "v"):
                code = s["cache"][name + "_codes"][pages, h]
                if name == "v":
                    code = code.transpose(2, 3).flatten(1, 2)
                code = code.flatten(0, 1) if name == "k" else code.reshape(-1, code.shape[-1])
                full = torch.empty((code.shape[0], d), dtype=f8, device=out.device)
                if case["bits"] == 8:
                    full.copy_(code)
                else:
                    full[:, 0::2], full[:, 1::2] = code % 16, code // 16
                zero = 2 ** (case["bits"] - 1) if case["sym"] else s["cache"][name + "_zeros"][pages, h].to(f8).view(-1, 1)
                side.append(((full - zero) * s["cache"][name + "_scales"][pages, h].to(f8).view(-1, 1))[:m])
            for j in range(g):
                logit = s["q"][at:at + n, h * g + j].to(f8) @ side[0].T / math.sqrt(d)
                out[at:at + n, h * g + j] = torch.softmax(logit.masked_fill(late, -math.inf), -1) @ side[1]
        at += n
    return {"out": out}
