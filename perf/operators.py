"""The measured cases of the operators around prefill attention, and their plain forms.

What a serving program does around the prefill attention of this package: rotate
q and k by their positions (``rope``), store k and v in a paged 8-bit cache
(``append``), attend over that cache one step at a time (``attention``), sum the
attention weight each key receives (``key_weights``), and drop the keys that
received least (``evict``).

With ``own`` false, ``run`` computes each operator with elementary torch
operations in 32 bits (angles in 64); with ``own`` true it makes the calls that a
user makes of the package. ``exact`` states each operator in 64 bits.

The cache: pages of ``page`` tokens, ``codes[num_pages, Hkv, page, D]`` in 8 bits
(int8 or e4m3) and ``range[num_pages, Hkv]`` in fp32; a code c of a block of range
r stands for c * r / F, F = 127 (int8) or 448 (e4m3).
"""
import math

import torch

own = False

HALF, INTERLEAVED = 0, 1
INT8, E4M3 = 0, 1
FULL = {INT8: 127.0, E4M3: 448.0}          # the code a block's range maps to
CODES = {INT8: torch.int8, E4M3: torch.float8_e4m3fn}


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch: a row of q and k per sequence at its own far position,
        # read out of the packed projection; latency counts
        dict(name="rope-step", op="rope", B=64, N=1, Hq=32, Hkv=8, D=128, rot=128, layout=HALF,
             positions=True, packed=True, factor=1.0),
        # a 128K prefill with frequencies scaled for long contexts: bandwidth counts
        dict(name="rope-prefill", op="rope", B=1, N=131072, Hq=32, Hkv=8, D=128, rot=128,
             layout=HALF, positions=False, packed=True, factor=8.0),
        # half of a small head in the interleaved layout, odd length, 7 q heads to a kv head
        dict(name="rope-part", op="rope", B=2, N=4173, Hq=28, Hkv=4, D=64, rot=32,
             layout=INTERLEAVED, positions=True, packed=False, factor=1.0),
        # one token of each sequence of a batch into the cache, mid-page; latency counts
        dict(name="append-step", op="append", B=64, n=1, Hkv=8, D=128, page=64, format=INT8,
             start=4000, ragged=False),
        # k and v of a whole 128K prompt into an empty cache: bandwidth counts
        dict(name="append-prefill", op="append", B=1, n=131072, Hkv=8, D=128, page=64, format=E4M3,
             start=0, ragged=False),
        # one sequence, a thousand tokens: the smallest decode, latency counts
        dict(name="attention-one", op="attention", B=1, nq=1, Hq=32, Hkv=8, D=128, page=64,
             format=INT8, most=1000, ragged=False, weights=False),
        # a serving batch of unequal lengths, small pages, 7 q heads to a kv head, with the
        # weight of each key for a later eviction
        dict(name="attention-batch", op="attention", B=24, nq=1, Hq=28, Hkv=4, D=128, page=16,
             format=E4M3, most=32768, ragged=True, weights=True),
        # long contexts, the whole card on one step: bandwidth counts
        dict(name="attention-long", op="attention", B=8, nq=1, Hq=32, Hkv=8, D=128, page=64,
             format=INT8, most=131072, ragged=False, weights=False),
        # weights of a 128K prompt's keys from its last 256 queries: tensor cores and exponentials
        dict(name="weights-prefill", op="weights", B=1, N=131072, Hq=32, Hkv=8, D=128, L=256,
             ragged=False),
        # a padded batch of short prompts, odd sizes, small heads
        dict(name="weights-batch", op="weights", B=2, N=4173, Hq=28, Hkv=4, D=64, L=100,
             ragged=True),
        # compress a 128K prompt as it is stored: choose 4096 keys a head, store only those
        dict(name="evict-prefill", op="evict", B=1, n=131072, Hkv=8, D=128, page=64, format=INT8,
             keep=4096, sinks=64, recent=256, ragged=False, cached=False),
        # shrink the caches of a running batch to a quarter, into fresh pages
        dict(name="evict-cache", op="evict", B=16, n=8192, Hkv=8, D=128, page=64, format=E4M3,
             keep=2048, sinks=16, recent=128, ragged=True, cached=True),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], its logarithm uniform."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "weights", "evict"])
    Hq, Hkv = rng.choice([(32, 8), (28, 4), (8, 1), (4, 4), (7, 1), (16, 2), (24, 8), (32, 2)])
    D = rng.choice([64, 128])
    page, fmt = rng.choice([16, 32, 64, 128]), rng.choice([INT8, E4M3])
    if op == "rope":
        N = _log(rng, 1, 131072)
        return dict(op=op, B=_log(rng, 1, max(1, min(64, 131072 // N))), N=N, Hq=Hq, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D // 2, D // 4, 2 * rng.randint(1, D // 2)]),
                    layout=rng.choice([HALF, INTERLEAVED]), positions=rng.random() < 0.5,
                    packed=rng.random() < 0.5, factor=rng.choice([1.0, 4.0, 8.0]))
    if op == "append":
        n = _log(rng, 1, 65536)
        return dict(op=op, B=_log(rng, 1, max(1, min(64, 65536 // n))), n=n, Hkv=Hkv, D=D,
                    page=page, format=fmt, start=rng.choice([0, _log(rng, 1, 4096)]),
                    ragged=rng.random() < 0.5)
    if op == "attention":
        most = _log(rng, 1, 131072)
        return dict(op=op, B=_log(rng, 1, max(1, min(64, (1 << 22) // (most * Hkv)))),
                    nq=rng.choice([1, 1, 1, 2, 3, 4, 8]), Hq=Hq, Hkv=Hkv, D=D, page=page,
                    format=fmt, most=most, ragged=rng.random() < 0.5, weights=rng.random() < 0.3)
    if op == "weights":
        N = _log(rng, 1, 131072)
        return dict(op=op, B=_log(rng, 1, max(1, min(8, 131072 // N))), N=N, Hq=Hq, Hkv=Hkv, D=D,
                    L=_log(rng, 1, min(N, 256)), ragged=rng.random() < 0.5)
    n = _log(rng, 16, 65536)
    keep = _log(rng, 8, n)
    sinks = min(rng.choice([0, 4, 64]), keep // 3)
    return dict(op=op, B=_log(rng, 1, max(1, min(32, 65536 // n))), n=n, Hkv=Hkv, D=D, page=page,
                format=fmt, keep=keep, sinks=sinks, recent=rng.randint(0, (keep - sinks) // 2),
                ragged=rng.random() < 0.5, cached=rng.random() < 0.5)


def work(case):
    c, D = case, case["D"]
    if c["op"] == "rope":
        rows = c["B"] * c["N"]
        return {"bytes": rows * (c["Hq"] + c["Hkv"]) * D * 4 + (rows * 4 if c["positions"] else 0),
                "flops": rows * (c["Hq"] + c["Hkv"]) * c["rot"] * 3}
    if c["op"] == "append":
        e = sum(_counts(c)) * c["Hkv"] * D * 2
        return {"bytes": e * 3, "flops": e * 3}
    if c["op"] == "attention":
        tok = sum(_lens(c))
        return {"bytes": tok * c["Hkv"] * (2 * D + (4 if c["weights"] else 0))
                + 4 * c["B"] * c["nq"] * c["Hq"] * D,
                "flops": 4 * tok * c["nq"] * c["Hq"] * D}
    if c["op"] == "weights":
        lens = _lens(dict(c, most=c["N"], nq=1))
        pairs = sum(min(c["L"], n) * n - min(c["L"], n) * (min(c["L"], n) - 1) // 2 for n in lens)
        return {"bytes": sum(lens) * c["Hkv"] * (2 * D + 4)
                + sum(min(c["L"], n) for n in lens) * c["Hq"] * D * 2,
                "flops": 2 * pairs * c["Hq"] * D}
    lens = _lens(dict(c, most=c["n"], nq=1))
    kept = sum(min(n, c["keep"]) for n in lens) * c["Hkv"]
    return {"bytes": sum(lens) * c["Hkv"] * 4 + kept * (4 + (8 if c["cached"] else 0)
                                                        + 2 * D * (2 if c["cached"] else 3)),
            "flops": sum(lens) * c["Hkv"] + kept * D * 4}


# ------------------------------------------------------------------------------ inputs

def _lens(c):
    """Tokens of each sequence. Ragged: from a hundredth of the most to the most, in a fixed mix."""
    B, most = c["B"], c["most"]
    if not c["ragged"]:
        return [most] * B
    return [most if b == 0 else max(1, int(most * 0.01 ** ((b * 0.6180339887) % 1.0)))
            for b in range(B)]


def _counts(c):
    """New tokens of each sequence of an append."""
    return _lens(dict(c, most=c["n"]))


def _pages(tokens, page):
    return (tokens + page - 1) // page


def _random(g, shape, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda") * scale


def _keys(g, B, N, H, D):
    """Keys as projections give them: a few channels several times larger than the others."""
    k = _random(g, (B, N, H, D), 1.0)
    k[..., :: max(1, D // 4)] *= 6.0
    return k.to(torch.bfloat16)


def _codes(g, shape, fmt):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
    if fmt == INT8:
        return x.mul_(32.0).round_().clamp_(-127, 127).to(torch.int8)
    return x.mul_(112.0).clamp_(-448, 448).to(torch.float8_e4m3fn)


def _bf16_ranges(g, shape, mid):
    r = mid * (0.6 + 0.8 * torch.rand(shape, generator=g, device="cuda"))
    return r.to(torch.bfloat16).float()


def _pool(g, s, pages, c):
    """A cache of `pages` pages, filled, and a table of all of them in random order."""
    H, P, D, fmt = c["Hkv"], c["page"], c["D"], c["format"]
    s["k8"], s["v8"] = _codes(g, (pages, H, P, D), fmt), _codes(g, (pages, H, P, D), fmt)
    s["k_range"], s["v_range"] = _bf16_ranges(g, (pages, H), 8.0), _bf16_ranges(g, (pages, H), 4.0)


def _table(g, s, B, per):
    order = torch.randperm(s["k8"].shape[0], generator=g, device="cuda")[: B * per]
    return order.to(torch.int32).view(B, per)


def _inv_freq(c):
    """Rotary frequencies; a factor above 1 divides the slow ones by it (long contexts)."""
    i = torch.arange(0, c["rot"], 2, dtype=torch.float64)
    f = 500000.0 ** (-i / c["rot"])
    if c["factor"] > 1.0:
        turns = 8192.0 * f / (2.0 * math.pi)
        smooth = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        f = f * (smooth + (1.0 - smooth) / c["factor"])
    return f.cuda()


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    s, D = {"case": dict(case)}, case["D"]
    op = c["op"]
    if op == "rope":
        B, N, Hq, Hkv = c["B"], c["N"], c["Hq"], c["Hkv"]
        width = (Hq + 2 * Hkv) * D if c["packed"] else None
        if c["packed"]:
            x = _random(g, (B, N, width), 2.0).to(torch.bfloat16)
            s["q"] = x[..., : Hq * D].unflatten(-1, (Hq, D))
            s["k"] = x[..., Hq * D: (Hq + Hkv) * D].unflatten(-1, (Hkv, D))
        else:
            s["q"] = _random(g, (B, N, Hq, D), 2.0).to(torch.bfloat16)
            s["k"] = _random(g, (B, N, Hkv, D), 2.0).to(torch.bfloat16)
        s["q_out"] = torch.empty((B, N, Hq, D), dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty((B, N, Hkv, D), dtype=torch.bfloat16, device="cuda")
        s["inv_freq"] = _inv_freq(c)
        s["mscale"] = 1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0
        s["first"] = 17
        s["positions"] = None
        if c["positions"]:
            begin = torch.randint(0, 131072, (B, 1), generator=g, device="cuda")
            s["positions"] = (begin + torch.arange(N, device="cuda")).to(torch.int32)
    elif op == "append":
        B, n = c["B"], c["n"]
        per = _pages(c["start"] + n, c["page"]) + 1
        _pool(g, s, B * per, c)
        s["table"] = _table(g, s, B, per)
        start = torch.randint(0, c["start"] + 1, (B,), generator=g, device="cuda")
        s["lens"] = start.to(torch.int32)
        s["counts"] = (torch.tensor(_counts(c), dtype=torch.int32, device="cuda")
                       if c["ragged"] else None)
        s["k"] = _keys(g, B, n, c["Hkv"], D)
        s["v"] = _random(g, (B, n, c["Hkv"], D)).to(torch.bfloat16)
    elif op == "attention":
        B, nq = c["B"], c["nq"]
        per = _pages(c["most"], c["page"])
        _pool(g, s, B * per, c)
        s["table"] = _table(g, s, B, per)
        s["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
        s["q"] = _random(g, (B, nq, c["Hq"], D), 1.0).to(torch.bfloat16)
        s["o"] = torch.empty_like(s["q"])
        s["scale"] = 1.0 / math.sqrt(D)
        s["weights"] = (torch.zeros((B, c["Hkv"], c["most"]), device="cuda")
                        if c["weights"] else None)
        if own:
            import long_context_prefill_trianglemix_b200 as tm
            size = tm.tm_kv8_attn_workspace_size(B, nq, c["Hq"], c["Hkv"], D, per, c["page"],
                                                 c["weights"])
            s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    elif op == "weights":
        B, N, Hq, Hkv = c["B"], c["N"], c["Hq"], c["Hkv"]
        s["q"] = _random(g, (B, N, Hq, D), 1.0).to(torch.bfloat16)
        s["k"] = _keys(g, B, N, Hkv, D)
        s["scale"] = 1.0 / math.sqrt(D)
        s["lens"] = (torch.tensor(_lens(dict(c, most=N)), dtype=torch.int32, device="cuda")
                     if c["ragged"] else None)
        s["weights"] = torch.zeros((B, Hkv, N), device="cuda")
        if own:
            import long_context_prefill_trianglemix_b200 as tm
            size = tm.tm_key_weights_workspace_size(B, Hq, Hkv, N, D, c["L"])
            s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    else:
        B, n, keep, P = c["B"], c["n"], c["keep"], c["page"]
        # accumulated weights: a heavy tail, and many keys that received nothing at all
        w = _random(g, (B, c["Hkv"], n), 2.0).exp_()
        w[torch.rand(w.shape, generator=g, device="cuda") < 0.2] = 0.0
        s["weights"] = w
        s["lens"] = torch.tensor(_lens(dict(c, most=n)), dtype=torch.int32, device="cuda")
        s["index"] = torch.full((B, c["Hkv"], keep), -1, dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros((B,), dtype=torch.int32, device="cuda")
        before, after = _pages(n, P), _pages(keep, P)
        if c["cached"]:
            _pool(g, s, B * (before + after), c)
            both = _table(g, s, B, before + after)
            s["table"], s["new_table"] = both[:, :before].contiguous(), both[:, before:].contiguous()
            s["new_weights"] = torch.zeros((B, c["Hkv"], keep), device="cuda")
        else:
            _pool(g, s, B * after, c)
            s["new_table"] = _table(g, s, B, after)
            s["empty"] = torch.zeros((B,), dtype=torch.int32, device="cuda")
            s["k"] = _keys(g, B, n, c["Hkv"], D)
            s["v"] = _random(g, (B, n, c["Hkv"], D)).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------------------ the passes

def run(state):
    return {"rope": _rope, "append": _append, "attention": _attention, "weights": _weights,
            "evict": _evict}[state["case"]["op"]](state)


def _rope(s):
    c = s["case"]
    q, k, D, rot = s["q"], s["k"], c["D"], c["rot"]
    if own:
        import long_context_prefill_trianglemix_b200 as tm
        tm.tm_rope_fwd(q, s["q_out"], k, s["k_out"], c["B"], c["N"], c["Hq"], c["Hkv"], D,
                       q.stride(1), c["Hq"] * D, k.stride(1), c["Hkv"] * D, rot, c["layout"], 0,
                       s["inv_freq"], s["mscale"], s["positions"], s["first"])
        return s["q_out"], s["k_out"]
    pos = s["positions"]
    if pos is None:
        pos = (s["first"] + torch.arange(c["N"], device="cuda")).expand(c["B"], -1)
    angle = pos.double().unsqueeze(-1) * s["inv_freq"]
    cos = (angle.cos() * s["mscale"]).float().unsqueeze(2)
    sin = (angle.sin() * s["mscale"]).float().unsqueeze(2)

    def turn(x):
        x = x.float()
        if c["layout"] == HALF:
            a, b = x[..., : rot // 2], x[..., rot // 2: rot]
            y = torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., rot:]), -1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2),
                           x[..., rot:]), -1)
        return y.to(torch.bfloat16)

    return turn(q), turn(k)


def _encode(x, r, fmt):
    """Codes of values x in a block of range r (broadcast): a zero range gives zeros."""
    y = torch.where(r > 0, x * FULL[fmt] / torch.where(r > 0, r, torch.ones_like(r)),
                    torch.zeros_like(x))
    return y.round().to(torch.int8) if fmt == INT8 else y.to(torch.float8_e4m3fn)


def _store(x, lens, counts, table, codes, ranges, c):
    """x [B, n, Hkv, D] into the cache behind lens[b] tokens: the blocks that it touches, as whole
    blocks [B, blocks, Hkv, page, D]."""
    B, n, H, D = x.shape
    P, fmt = c["page"], c["format"]
    first = lens.long() // P
    block = first[:, None] + torch.arange((n - 1) // P + 2, device=x.device)
    slot = block[..., None] * P + torch.arange(P, device=x.device)
    token = slot - lens.long()[:, None, None]
    new = (token >= 0) & (token < counts.long()[:, None, None])
    old = token < 0
    at = token.clamp(0, n - 1).flatten(1)
    y = torch.gather(x.float(), 1, at[..., None, None].expand(-1, -1, H, D))
    y = y.unflatten(1, slot.shape[1:]).transpose(2, 3)          # [B, blocks, H, P, D]
    new, old = new[:, :, None, :, None], old[:, :, None, :, None]
    y = torch.where(new, y, torch.zeros_like(y))
    pages = table.long().gather(1, block.clamp(max=table.shape[1] - 1))
    cur, r0 = codes.view(torch.int8)[pages].view(codes.dtype), ranges[pages][..., None, None]
    r0 = torch.where(old.any(3, keepdim=True), r0, torch.zeros_like(r0))
    r = torch.maximum(r0, y.abs().amax((3, 4), keepdim=True))
    moved = torch.where(r > 0, cur.float() * r0 / torch.where(r > 0, r, torch.ones_like(r)), 0.0)
    moved = moved.round().to(torch.int8) if fmt == INT8 else moved.to(torch.float8_e4m3fn)
    out = torch.where(new, _encode(y, r, fmt).view(torch.int8),
                      torch.where(old, moved.view(torch.int8), cur.view(torch.int8)))
    touched = new.any(3).flatten(2).any(2)
    codes.view(torch.int8)[pages[touched]] = out[touched]
    ranges[pages[touched]] = r[touched][..., 0, 0]


def _append(s):
    c = s["case"]
    if own:
        import long_context_prefill_trianglemix_b200 as tm
        tm.tm_kv8_append(s["k"], s["v"], s["k"].stride(1), s["v"].stride(1), c["B"], c["n"], c["n"],
                         c["Hkv"], c["D"], s["counts"], None, s["lens"], s["table"],
                         s["table"].shape[1], s["k8"], s["v8"], s["k_range"], s["v_range"],
                         s["k8"].shape[0], c["page"], c["format"])
    else:
        counts = s["counts"]
        if counts is None:
            counts = torch.full((c["B"],), c["n"], device="cuda")
        _store(s["k"], s["lens"], counts, s["table"], s["k8"], s["k_range"], c)
        _store(s["v"], s["lens"], counts, s["table"], s["v8"], s["v_range"], c)
    return s["k8"], s["v8"], s["k_range"], s["v_range"]


def _read(codes, ranges, table, c, most):
    """The values of the cache, [B, Hkv, most, D]."""
    x = codes.view(torch.int8)[table.long()].view(codes.dtype).float()
    x = x * (ranges[table.long()] / FULL[c["format"]])[..., None, None]
    return x.transpose(1, 2).flatten(2, 3)[:, :, :most]


def _attention(s):
    c = s["case"]
    B, nq, Hq, Hkv, D, most = c["B"], c["nq"], c["Hq"], c["Hkv"], c["D"], c["most"]
    if own:
        import long_context_prefill_trianglemix_b200 as tm
        tm.tm_kv8_attn_fwd(s["q"], s["o"], B, nq, Hq, Hkv, D, s["scale"], s["k8"], s["v8"],
                           s["k_range"], s["v_range"], s["k8"].shape[0], c["page"], c["format"],
                           s["table"], s["table"].shape[1], s["lens"], s["weights"], most, 0,
                           s["workspace"], s["workspace"].numel())
        return (s["o"], s["weights"]) if c["weights"] else s["o"]
    k = _read(s["k8"], s["k_range"], s["table"], c, most)
    v = _read(s["v8"], s["v_range"], s["table"], c, most)
    q = s["q"].float().view(B, nq, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = torch.matmul(q, k.transpose(2, 3)) * s["scale"]     # [B, Hkv, nq G, most]
    row = torch.arange(nq * (Hq // Hkv), device="cuda") // (Hq // Hkv)
    last = s["lens"].long()[:, None] - nq + row                 # last key of each row
    seen = torch.arange(most, device="cuda") <= last[..., None]
    score = torch.where(seen[:, None], score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    o = torch.matmul(p, v).view(B, Hkv, nq, Hq // Hkv, D).permute(0, 2, 1, 3, 4)
    o = o.reshape(B, nq, Hq, D).to(torch.bfloat16)
    return (o, p.sum(2)) if c["weights"] else o


def _weights(s):
    c = s["case"]
    B, N, Hq, Hkv, D, L = c["B"], c["N"], c["Hq"], c["Hkv"], c["D"], c["L"]
    if own:
        import long_context_prefill_trianglemix_b200 as tm
        tm.tm_key_weights_fwd(s["q"], s["k"], B, Hq, Hkv, N, D, s["scale"], L, s["lens"],
                              s["weights"], N, 0, s["workspace"], s["workspace"].numel())
        return s["weights"]
    lens = s["lens"]
    if lens is None:
        lens = torch.full((B,), N, device="cuda")
    row = lens.long()[:, None] - L + torch.arange(L, device="cuda")      # [B, L]
    at = row.clamp(min=0)[..., None, None].expand(-1, -1, Hq, D)
    q = torch.gather(s["q"], 1, at).float().view(B, L, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    k = s["k"].float().permute(0, 2, 3, 1)                               # [B, Hkv, D, N]
    score = torch.matmul(q.flatten(2, 3), k).unflatten(2, (Hq // Hkv, L)) * s["scale"]
    seen = (torch.arange(N, device="cuda") <= row[..., None])[:, None, None]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    return (p / torch.where(total > 0, total, torch.ones_like(total))).sum((2, 3))


def _select(s):
    c = s["case"]
    B, n, keep = c["B"], c["n"], c["keep"]
    lens = s["lens"].long()[:, None, None]
    at = torch.arange(n, device="cuda")
    kept = lens.clamp(max=keep)
    held = (at < c["sinks"]) | (at >= lens - c["recent"])
    w = torch.where(held, torch.full_like(s["weights"], math.inf), s["weights"])
    w = torch.where(at < lens, w, torch.full_like(w, -math.inf))
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    take = torch.arange(keep, device="cuda")
    order = torch.where(take < kept, order, torch.full_like(order, n)).sort(-1).values
    index = torch.where(take < kept, order, torch.full_like(order, -1)).to(torch.int32)
    return index, kept.flatten().to(torch.int32)


def _move(codes, ranges, table, new_table, index, kept, c):
    """The kept tokens' codes into the pages of new_table, each block at its sources' largest range."""
    P, fmt, H = c["page"], c["format"], c["Hkv"]
    B, keep = index.shape[0], index.shape[2]
    blocks = new_table.shape[1]
    at = torch.nn.functional.pad(index.long(), (0, blocks * P - keep), value=-1)
    live = at >= 0
    at = at.clamp(min=0)
    page = table.long().gather(1, (at // P).flatten(1)).view_as(at)      # [B, H, blocks P]
    head = torch.arange(H, device="cuda")[None, :, None].expand_as(page)
    x = codes.view(torch.int8)[page, head, at % P].view(codes.dtype).float()
    r1 = torch.where(live, ranges[page, head], torch.zeros_like(page, dtype=torch.float32))
    r1 = r1.unflatten(2, (blocks, P))
    r2 = r1.amax(3)
    y = x.unflatten(2, (blocks, P)) * r1[..., None]
    y = torch.where(r2[..., None, None] > 0,
                    y / torch.where(r2 > 0, r2, torch.ones_like(r2))[..., None, None], 0.0)
    y = (y.round().to(torch.int8) if fmt == INT8 else y.to(torch.float8_e4m3fn)).view(torch.int8)
    y, r2 = y.transpose(1, 2), r2.transpose(1, 2)                        # [B, blocks, H, ...]
    live = live.unflatten(2, (blocks, P)).transpose(1, 2)
    to = new_table.long()
    codes.view(torch.int8)[to] = torch.where(live[..., None], y, codes.view(torch.int8)[to])
    ranges[to] = torch.where(live.any(3), r2, ranges[to])


def _evict(s):
    c = s["case"]
    B, n, keep, H, D, P = c["B"], c["n"], c["keep"], c["Hkv"], c["D"], c["page"]
    if own:
        import long_context_prefill_trianglemix_b200 as tm
        tm.tm_kv_select(s["weights"], n, s["lens"], B, H, n, keep, c["sinks"], c["recent"],
                        s["index"], s["kept"])
        if c["cached"]:
            tm.tm_kv8_compact(s["index"], keep, s["kept"], s["lens"], B, H, D, s["table"],
                              s["table"].shape[1], s["new_table"], s["new_table"].shape[1], s["k8"],
                              s["v8"], s["k_range"], s["v_range"], s["k8"].shape[0], P, c["format"],
                              s["weights"], n, s["new_weights"], keep)
        else:
            tm.tm_kv8_append(s["k"], s["v"], s["k"].stride(1), s["v"].stride(1), B, n, keep, H, D,
                             s["kept"], s["index"], s["empty"], s["new_table"],
                             s["new_table"].shape[1], s["k8"], s["v8"], s["k_range"], s["v_range"],
                             s["k8"].shape[0], P, c["format"])
        return ((s["index"], s["kept"], s["k8"], s["v8"], s["k_range"], s["v_range"])
                + ((s["new_weights"],) if c["cached"] else ()))
    index, kept = _select(s)
    more = ()
    if c["cached"]:
        _move(s["k8"], s["k_range"], s["table"], s["new_table"], index, kept, c)
        _move(s["v8"], s["v_range"], s["table"], s["new_table"], index, kept, c)
        picked = s["weights"].gather(2, index.long().clamp(min=0))
        more = (torch.where(index >= 0, picked, s["new_weights"]),)
    else:
        at = index.long().clamp(min=0).transpose(1, 2)[..., None].expand(-1, -1, -1, D)
        _store(s["k"].gather(1, at), s["empty"], kept, s["new_table"], s["k8"], s["k_range"], c)
        _store(s["v"].gather(1, at), s["empty"], kept, s["new_table"], s["v8"], s["v_range"], c)
    return (index, kept, s["k8"], s["v8"], s["k_range"], s["v_range"]) + more


# ------------------------------------------------------------------------------ in 64 bits

def _nearest(y, fmt):
    """y rounded to the nearest code, ties to even, in 64 bits."""
    if fmt == INT8:
        return torch.round(y)
    a = y.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6.0) - 3.0)
    return torch.sign(y) * torch.clamp(torch.round(a / step) * step, max=448.0)


def _values(codes):
    return codes.to(torch.float64) if codes.dtype == torch.int8 else codes.float().double()


def _exact_append(k, lens, counts, table, codes, ranges, c):
    """Token by token's definition, one block of one sequence at a time."""
    P, fmt = c["page"], c["format"]
    out, new = _values(codes), ranges.double().clone()
    lens, counts, table = lens.tolist(), counts.tolist(), table.tolist()
    for b in range(len(lens)):
        a, e = lens[b], lens[b] + counts[b]
        whole = [] if e <= a else range(a // P, (e - 1) // P + 1)
        inner = [j for j in whole if j * P >= a and (j + 1) * P <= e]
        if inner:
            x = k[b, inner[0] * P - a: (inner[-1] + 1) * P - a].double()
            x = x.unflatten(0, (len(inner), P)).transpose(1, 2)
            r = x.abs().amax((2, 3))
            y = torch.where(r[..., None, None] > 0, x * FULL[fmt] / r[..., None, None], 0.0)
            pages = torch.tensor([table[b][j] for j in inner], device="cuda")
            out[pages], new[pages] = _nearest(y, fmt), r
        for j in (j for j in whole if j not in inner):
            lo, hi, p = max(a, j * P), min(e, (j + 1) * P), table[b][j]
            x = k[b, lo - a: hi - a].double().transpose(0, 1)
            before = new[p] if lo > j * P else torch.zeros_like(new[p])
            r = torch.maximum(before, x.abs().amax((1, 2)))
            d = torch.where(r > 0, r, torch.ones_like(r))[:, None, None]
            out[p][:, : lo - j * P] = _nearest(out[p][:, : lo - j * P] * before[:, None, None] / d, fmt)
            out[p][:, lo - j * P: hi - j * P] = _nearest(x * FULL[fmt] / d, fmt)
            new[p] = r
    return (out.long() if fmt == INT8 else out), new


def exact(case, seed):
    c, s = case, prepare(case, seed)
    D, op = c["D"], case["op"]
    if op == "rope":
        pos = s["positions"]
        if pos is None:
            pos = torch.arange(s["first"], s["first"] + c["N"], device="cuda").expand(c["B"], -1)
        turn = torch.polar(torch.full((), s["mscale"], dtype=torch.float64, device="cuda"),
                           (pos.double()[..., None] * s["inv_freq"])[:, :, None])
        out = []
        for x in (s["q"], s["k"]):
            y = x.double().contiguous()
            r = y[..., : c["rot"]].unflatten(-1, (2, -1) if c["layout"] == HALF else (-1, 2))
            r = r.transpose(-1, -2) if c["layout"] == HALF else r
            z = torch.view_as_real(torch.view_as_complex(r.contiguous()) * turn)
            z = z.transpose(-1, -2) if c["layout"] == HALF else z
            y[..., : c["rot"]] = z.flatten(-2)
            out.append(y)
        return tuple(out)
    if op == "append":
        counts = s["counts"]
        if counts is None:
            counts = torch.full((c["B"],), c["n"])
        k8, kr = _exact_append(s["k"], s["lens"], counts, s["table"], s["k8"], s["k_range"], c)
        v8, vr = _exact_append(s["v"], s["lens"], counts, s["table"], s["v8"], s["v_range"], c)
        return k8, v8, kr, vr
    if op == "attention":
        B, nq, Hq, Hkv, G = c["B"], c["nq"], c["Hq"], c["Hkv"], c["Hq"] // c["Hkv"]
        o = torch.zeros((B, nq, Hq, D), dtype=torch.float64, device="cuda")
        w = torch.zeros((B, Hkv, c["most"]), dtype=torch.float64, device="cuda")
        full = FULL[c["format"]]
        for b, n in enumerate(s["lens"].tolist()):
            pages = s["table"][b, : _pages(n, c["page"])].long()
            for h in range(Hkv):
                k = _values(s["k8"].view(torch.int8)[pages, h].view(s["k8"].dtype))
                v = _values(s["v8"].view(torch.int8)[pages, h].view(s["v8"].dtype))
                k = (k * s["k_range"][pages, h].double()[:, None, None] / full).flatten(0, 1)[:n]
                v = (v * s["v_range"][pages, h].double()[:, None, None] / full).flatten(0, 1)[:n]
                for i in range(max(0, nq - n), nq):
                    seen = n - nq + i + 1
                    heads = slice(h * G, (h + 1) * G)
                    p = torch.softmax(s["q"][b, i, heads].double() @ k[:seen].T * s["scale"], -1)
                    o[b, i, heads] = p @ v[:seen]
                    w[b, h, :seen] += p.sum(0)
        return (o, w) if c["weights"] else o
    if op == "weights":
        B, N, Hq, Hkv, G = c["B"], c["N"], c["Hq"], c["Hkv"], c["Hq"] // c["Hkv"]
        lens = [N] * B if s["lens"] is None else s["lens"].tolist()
        w = torch.zeros((B, Hkv, N), dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            rows = torch.arange(max(0, n - c["L"]), n, device="cuda")
            ahead = torch.arange(n, device="cuda") > rows[:, None]
            for h in range(Hq):
                k = s["k"][b, :n, h // G].double()
                score = (s["q"][b, rows, h].double() @ k.T) * s["scale"]
                w[b, h // G, :n] += torch.softmax(score.masked_fill(ahead, -math.inf), -1).sum(0)
        return w
    B, H, n, keep, P = c["B"], c["Hkv"], c["n"], c["keep"], c["page"]
    index = torch.full((B, H, keep), -1, dtype=torch.int64, device="cuda")
    kept = []
    for b, m in enumerate(s["lens"].tolist()):
        for h in range(H):
            w = s["weights"][b, h, :m].double().cpu().numpy()
            key = sorted(range(m), key=lambda j, w=w, m=m: (
                not (j < c["sinks"] or j >= m - c["recent"]), -w[j], j))[: min(m, keep)] \
                if m <= 16384 else _top(s["weights"][b, h, :m].double(), m, c)
            index[b, h, : min(m, keep)] = torch.tensor(sorted(key), device="cuda")
        kept.append(min(m, keep))
    if not c["cached"]:
        out = []
        for x, codes, ranges in ((s["k"], s["k8"], s["k_range"]), (s["v"], s["v8"], s["v_range"])):
            at = index.clamp(min=0).transpose(1, 2)[..., None].expand(-1, -1, -1, D)
            out += _exact_append(x.gather(1, at), s["empty"], torch.tensor(kept), s["new_table"],
                                 codes, ranges, c)
        return index, torch.tensor(kept), out[0], out[2], out[1], out[3]
    out = []
    for codes, ranges in ((s["k8"], s["k_range"]), (s["v8"], s["v_range"])):
        x, r = _values(codes), ranges.double().clone()
        src, rs = x.clone(), r.clone()
        for b in range(B):
            for j in range(_pages(kept[b], P)):
                slots = index[b, :, j * P: min(kept[b], (j + 1) * P)]        # [H, tokens]
                page, head = s["table"][b].long()[slots // P], torch.arange(H, device="cuda")[:, None]
                r1 = rs[page, head]
                r2 = r1.amax(1)
                to = int(s["new_table"][b, j])
                y = src[page, head, slots % P] * r1[..., None] / r2[:, None, None]
                x[to][:, : slots.shape[1]] = _nearest(y, c["format"])
                r[to] = r2
        out += [x.long() if c["format"] == INT8 else x, r]
    picked = torch.zeros((B, H, keep), dtype=torch.float64, device="cuda")
    for b in range(B):
        picked[b, :, : kept[b]] = s["weights"][b].double().gather(1, index[b, :, : kept[b]])
    return index, torch.tensor(kept), out[0], out[2], out[1], out[3], picked


def _top(w, m, c):
    """The kept keys of one long row: the protected ones, then those above the border, then the
    first of those at it."""
    at = torch.arange(m, device=w.device)
    held = (at < c["sinks"]) | (at >= m - c["recent"])
    left = min(m, c["keep"]) - int(held.sum())
    rest = w[~held]
    if left <= 0:
        return at[held].tolist()
    border = rest.sort(descending=True).values[left - 1]
    above = ~held & (w > border)
    level = at[~held & (w == border)][: left - int(above.sum())]
    return torch.cat((at[held | above], level)).tolist()
