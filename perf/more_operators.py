"""Measured cases of the target's serving step around a cache held in 4 bits: page tables and slot
maps from request lengths, norms of query and key heads with the position rotation, append to and
attention over a 4-bit paged cache, and log probabilities of given tokens.

The 4-bit cache: the D values of a slot's head in groups of 16.  A group has a scale s, an e4m3
number (4 bits exponent, 3 bits fraction) that is its largest magnitude / 6 rounded to nearest, at
most 448; a value is kept as the e2m1 number (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives) nearest
to value / s, ties to the even code.  Pools: codes uint8 [pages, KV heads, page size, D/2], two
values a byte, the even one in the low half; scales [pages, KV heads, page size, D/16].
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _case(op, name=None, **kw):
    c = dict(op=op, **kw)
    if name:
        c["name"] = name
    return c


def _paged(op, name=None, *, dtype="bf16", B, hkv=8, group=4, d=128, page=64, lo, hi, rlo, rhi, window=0, sinks=0, lens=1):
    """lo..hi: slots held by a request; rlo..rhi: its new rows; lens: what the lengths are drawn from."""
    return _case(op, name, dtype=dtype, B=B, hkv=hkv, group=group, d=d, page=page, lo=lo, hi=hi, rlo=rlo, rhi=rhi, window=window,
                 sinks=sinks, lens=lens)


def _plan(name=None, *, B, page=64, lo, hi, rlo, rhi, short=0, give=True, lens=1):
    """lo..hi: slots that a request keeps; rlo..rhi: its new rows; short: pages that the step lacks."""
    return _case("plan", name, B=B, page=page, lo=lo, hi=hi, rlo=rlo, rhi=rhi, short=short, give=give, lens=lens)


def _heads(name=None, *, rows, hq=32, hkv=8, d=128, rotary=128, interleaved=False, dtype="bf16", far=32768):
    return _case("heads", name, rows=rows, hq=hq, hkv=hkv, d=d, rotary=rotary, interleaved=interleaved, dtype=dtype, far=far)


def _logprobs(name=None, *, rows, vocab=151936, dtype="fp32", top=8, given=1, temperature=1.0):
    return _case("logprobs", name, rows=rows, vocab=vocab, dtype=dtype, top=top, given=given, temperature=temperature)


def listed():
    return [
        # eight requests get the pages and slots of a drafted block of sixteen rows
        _plan("plan_block_b8", B=8, lo=512, hi=16384, rlo=16, rhi=16),
        # a large step: tokens and prompt chunks of 512 requests, small pages, pages of dropped rows given back
        _plan("plan_step_b512", B=512, page=16, lo=0, hi=32768, rlo=1, rhi=255, lens=2),
        # query and key heads of one token of each of eight requests (32 / 8 heads)
        _heads("heads_token_b8", rows=8),
        # a prompt's heads, half of each rotated, in pairs side by side
        _heads("heads_chunk", rows=8191, rotary=64, interleaved=True, dtype="fp16"),
        # the rows of eight verified blocks go into the cache
        _paged("append", "append4_block_b8", B=8, lo=512, hi=16384, rlo=16, rhi=16),
        # ragged prompt chunks of four requests, small pages
        _paged("append", "append4_chunk_b4", dtype="fp16", B=4, page=16, lo=8192, hi=9001, rlo=2048, rhi=8191, lens=2),
        # one new token of one request at the 27B geometry's context
        _paged("attend", "attend4_b1_4096", B=1, lo=4096, hi=4096, rlo=1, rhi=1),
        # one new token for each of sixteen long, ragged contexts
        _paged("attend", "attend4_b16_long", dtype="fp16", B=16, page=16, lo=4096, hi=32768, rlo=1, rhi=1, lens=3),
        # a drafted block of sixteen rows is verified for eight requests
        _paged("attend", "attend4_verify_b8", B=8, lo=512, hi=16384, rlo=16, rhi=16, lens=5),
        # a whole prompt of 8192 tokens, full attention
        _paged("attend", "attend4_prompt_8192", B=1, lo=8192, hi=8192, rlo=8192, rhi=8192),
        # one new token of each of eight requests: its log probability and eight alternatives
        _logprobs("logprobs_token_b8", rows=8),
        # the log probabilities of a prompt's tokens, twenty alternatives each
        _logprobs("logprobs_prompt", rows=2047, dtype="bf16", top=20, temperature=0.7),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    """One case of the same ranges: 1 to 512 requests, lengths 1 to 32768, blocks of 1 to 16 rows or
    prompt chunks of up to 8192, one to eight KV heads, groups of one to eight, pages of 8 to 256 slots
    (odd ones too), with and without a window; vocabularies of 1000 to 152000."""
    op = rng.choice(["plan", "heads", "append", "attend", "attend", "attend", "logprobs"])
    page = rng.choice([8, 16, 24, 32, 33, 64, 128, 256])
    lens = rng.randrange(10, 1 << 20)
    if op == "plan":
        B = _log(rng, 1, 512)
        hi, rhi = _log(rng, 1, 32768), _log(rng, 1, 255)
        return _plan(B=B, page=max(16, page), lo=int(hi * rng.uniform(0, 1)), hi=hi, rlo=rng.choice([0, 1, rhi]), rhi=rhi,
                     short=rng.choice([0, 0, 1, 7]), give=rng.random() < 0.7, lens=lens)
    if op == "heads":
        d = rng.choice([64, 128, 128, 256])
        rows, hkv = _log(rng, 1, 8191), rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
        rows = max(1, min(rows, 8191 * 40 * 128 // ((hq + hkv) * d)))
        return _heads(rows=rows, hq=hq, hkv=hkv, d=d, rotary=rng.choice([d, d, d // 2, d // 4]), interleaved=rng.random() < 0.4,
                      dtype=rng.choice(["bf16", "fp16"]), far=rng.choice([4096, 32768, 1 << 20]))
    if op == "logprobs":
        vocab, dtype = _log(rng, 1000, 152000), rng.choice(["fp32", "bf16", "fp16"])
        rows = min(_log(rng, 1, 2047), (2047 * 151936 * 2) // (vocab * (4 if dtype == "fp32" else 2)))
        return _logprobs(rows=max(1, rows), vocab=vocab, dtype=dtype, top=rng.choice([0, 1, 5, 8, 20]), given=rng.choice([1, 1, 2, 5]),
                         temperature=rng.choice([1.0, 0.7, 1.3]))
    heads = dict(hkv=rng.choice([1, 2, 4, 8]), group=rng.choice([1, 2, 3, 4, 5, 8]), d=rng.choice([64, 128, 128]),
                 dtype=rng.choice(["bf16", "fp16"]), page=page, lens=lens)
    win = dict(window=_log(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 17, 128])) if rng.random() < 0.4 else {}
    B = rng.choice([1, 1, 2, 3, 4, 5, 8, 12, 16])
    hi = _log(rng, 1, 32768)
    lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
    if op == "append":
        rhi = min(hi, _log(rng, 1, 8192))
        B = max(1, min(B, 65536 // hi))
        return _paged(op, B=B, lo=max(lo, rhi), hi=hi, rlo=max(1, int(rhi * rng.uniform(0.2, 1.0))), rhi=rhi, **heads)
    if rng.random() < 0.4:  # prompt chunks; no more score entries than the largest listed case has
        rhi = min(hi, _log(rng, 17, 8192))
        B = max(1, min(B, (1 << 30) // (heads["hkv"] * heads["group"] * hi * rhi), 65536 // hi))
    else:  # tokens and blocks
        rhi = min(hi, rng.choice([1, 1, 2, 3, 5, 7, 8, 13, 16]))
    return _paged(op, B=B, lo=max(lo, rhi), hi=hi, rlo=max(1, rhi - rng.randrange(0, 1 + rhi // 2)), rhi=rhi, **heads, **win)


def _lengths(c):
    r = random.Random(c["lens"])
    n = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    if c["op"] == "plan":
        return n, [r.randint(c["rlo"], c["rhi"]) for _ in n]
    return n, [r.randint(min(c["rlo"], x), min(c["rhi"], x)) for x in n]


def _pages(c):
    """Of a planning case: slots kept, new rows, pages held before (the last step's dropped rows may
    have left more than are needed, a request's growth fewer), entries of a table row, pages needed."""
    n, r = _lengths(c)
    g, ps = random.Random(c["lens"] + 1), c["page"]
    held = [max(0, -(-x // ps) + g.choice([0, 0, 0, 1])) for x in n]
    need = [-(-(x + y) // ps) for x, y in zip(n, r)]
    return n, r, held, max(max(held), max(need), 1), need


def _pairs(n, r, window, sinks):
    """(slots visible to some row, visible pairs) of r rows at the end of n slots."""
    if not r:
        return 0, 0
    p = np.arange(n - r, n, dtype=np.int64)
    if not window:
        return int(p[-1]) + 1, int((p + 1).sum())
    first = np.maximum(0, p - window + 1)
    seen = int(p[-1]) + 1 - int(first[0]) + min(sinks, int(first[0]))
    return seen, int((p + 1 - first + np.minimum(sinks, first)).sum())


def work(c):
    if c["op"] == "plan":
        n, r, held, _, need = _pages(c)
        moved = sum(abs(a - b) for a, b in zip(held, need) if a < b or c["give"])
        # lengths, counts and pages in; lengths, places, the rows' positions, requests and slots out
        touched = sum(-(-(x + y) // c["page"]) - x // c["page"] for x, y in zip(n, r))
        return {"bytes": 4 * 3 * c["B"] + 4 * 3 * c["B"] + 8 * moved + 4 * touched + 16 * sum(r), "flops": 0}
    if c["op"] == "heads":
        x = c["rows"] * (c["hq"] + c["hkv"]) * c["d"]
        return {"bytes": 4 * x + 4 * c["rows"], "flops": 8 * x}
    if c["op"] == "logprobs":
        x = c["rows"] * c["vocab"]
        return {"bytes": x * (4 if c["dtype"] == "fp32" else 2) + c["rows"] * (8 + 8 * c["given"] + 8 * c["top"]), "flops": 6 * x}
    n, r = _lengths(c)
    hq, hkv, d = c["hkv"] * c["group"], c["hkv"], c["d"]
    rows, kv = sum(r), hkv * d * 9 // 16  # one slot's keys: half a byte a value and a byte each 16
    table = 4 * sum(-(-x // c["page"]) for x in n)
    if c["op"] == "append":
        return {"bytes": 2 * rows * (2 * hkv * d + kv + 2 * hkv * d) + 4 * rows, "flops": 0}
    seen, pairs = (sum(v) for v in zip(*(_pairs(a, b, c["window"], c["sinks"]) for a, b in zip(n, r))))
    return {"bytes": 2 * seen * kv + rows * hq * (4 * d + 4) + table, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ the 4-bit form
def _encode(x):
    """Values [..., D] -> codes uint8 [..., D/2], scales e4m3 [..., D/16]."""
    x = x.float().unflatten(-1, (-1, 16))
    scale = (x.abs().amax(-1) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float()[..., None]
    y = torch.where(s > 0, x.abs() / s, 0.0)
    # the nearest of GRID; a tie goes to the even code
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = torch.where((s > 0) & torch.signbit(x), code + 8, code).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, scale


def _decode(codes, scales, t=torch.float32):
    """The values that codes and scales stand for."""
    grid = torch.tensor(GRID + [-v for v in GRID], device=codes.device, dtype=t)
    x = torch.stack((grid[(codes & 15).long()], grid[(codes >> 4).long()]), -1).flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * scales.to(t)[..., None]).flatten(-2)


# ------------------------------------------------------------------ inputs
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"plan": _prepare_plan, "heads": _prepare_heads, "logprobs": _prepare_logprobs}.get(c["op"], _prepare_paged)(c, g)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_plan(c, g):
    n, r, held, width, need = _pages(c)
    B, dev = c["B"], "cuda"
    rows = sum(r) + 13  # a captured step's row arrays are longer than a step's rows
    gained = sum(max(0, b - a) for a, b in zip(held, need))
    given = sum(max(0, a - b) for a, b in zip(held, need)) if c["give"] else 0
    free = max(0, gained - given - c["short"]) if c["short"] else max(0, gained - given) + 5
    total = sum(held) + free + 3
    ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device=dev)
    at = torch.arange(width, device=dev)[None] < _ints(held)[:, None]
    table[at] = ids[:sum(held)]
    stack = torch.full((total,), -1, dtype=torch.int32, device=dev)
    stack[:free] = ids[sum(held):sum(held) + free]
    z = lambda *shape, t=torch.int32: torch.full(shape, -7, dtype=t, device=dev)  # noqa: E731
    s = dict(c, len=_ints(n), new=_ints(r), held=_ints(held), table=table, stack=stack, free=_ints([free]), rows=rows, seq_len=z(B),
             row_start=z(B + 1), request=z(rows), pos=z(rows), slot=z(rows, t=torch.int64), held_out=z(B), free_out=z(1), n_short=z(1))
    if own:
        from block_drafter_gb300.paged import PageTables
        s["pages"] = PageTables(table, s["held"], stack, s["free"], c["page"], held_out=s["held_out"], free_count_out=s["free_out"])
    return s


def _prepare_heads(c, g):
    t, dev, d = TYPES[c["dtype"]], "cuda", c["d"]
    rows, hq, hkv = c["rows"], c["hq"], c["hkv"]
    # the projections' output: queries, keys and values side by side; gains near one
    qkv = (torch.randn(rows, hq + 2 * hkv, d, generator=g, device=dev) * 3.0).to(t)
    gain = lambda: (1 + 0.1 * torch.randn(d, generator=g, device=dev)).to(t)  # noqa: E731
    half = c["rotary"] // 2
    freq = torch.tensor([10000000.0 ** (-j / half) for j in range(half)], dtype=torch.float64, device=dev)
    s = dict(c, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], q_gain=gain(), k_gain=gain(), freq=freq,
             pos=torch.randint(0, c["far"], (rows,), generator=g, device=dev, dtype=torch.int32),
             q_out=torch.zeros(rows, hq, d, dtype=t, device=dev), k_out=torch.zeros(rows, hkv, d, dtype=t, device=dev))
    if own:
        from block_drafter_gb300.target import HeadNormRope
        s["op_"] = HeadNormRope(d, freq, s["q_gain"], s["k_gain"], eps=EPS, interleaved=c["interleaved"])
    return s


def _prepare_logprobs(c, g):
    t, dev, rows, vocab = TYPES[c["dtype"]], "cuda", c["rows"], c["vocab"]
    # a trained head's logits: a wide body, a few tokens far above it, and the given one among them or not
    logits = torch.randn(rows, vocab, generator=g, device=dev) * 2.5
    peaks = torch.randint(0, vocab, (rows, 24), generator=g, device=dev)
    logits.scatter_(1, peaks, torch.rand(rows, 24, generator=g, device=dev) * 12.0 + 6.0)
    tokens = torch.randint(0, vocab, (rows, c["given"]), generator=g, device=dev)
    tokens = torch.where(torch.rand(rows, c["given"], generator=g, device=dev) < 0.7, peaks[:, :c["given"]], tokens).to(torch.int32)
    return dict(c, logits=logits.to(t), tokens=tokens, logprob=torch.zeros(rows, c["given"], device=dev), entropy=torch.zeros(rows, device=dev),
                lse=torch.zeros(rows, device=dev), ids=torch.zeros(rows, max(1, c["top"]), dtype=torch.int32, device=dev),
                alt=torch.zeros(rows, max(1, c["top"]), device=dev))


def _prepare_paged(c, g):
    t, dev = TYPES[c["dtype"]], "cuda"
    n, r = _lengths(c)
    B, hkv, hq, d, ps = c["B"], c["hkv"], c["hkv"] * c["group"], c["d"], c["page"]
    held = [-(-x // ps) for x in n]
    cols, total = max(held), sum(held)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std).to(t)

    def pool():  # filled some pages at a time: the 32-bit values of a whole pool are eight times its size
        codes = torch.empty(total, hkv, ps, d // 2, dtype=torch.uint8, device=dev)
        scales = torch.empty(total, hkv, ps, d // 16, dtype=torch.float8_e4m3fn, device=dev)
        step = max(1, (1 << 26) // (hkv * ps * d))
        for i in range(0, total, step):
            codes[i:i + step], scales[i:i + step] = _encode(normal(min(step, total - i), hkv, ps, d))
        return codes, scales

    ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)  # pages lie anywhere in the pool
    table = torch.zeros(B, cols, dtype=torch.int32, device=dev)
    table[torch.arange(cols, device=dev)[None] < _ints(held)[:, None]] = ids
    rows = sum(r)
    s = dict(c, total=total, cols=cols, n=_ints(n), max_len=max(n), max_rows=max(r), start=_ints([0] + list(np.cumsum(r))), table=table,
             rows=rows, scale=1.0 / math.sqrt(d))
    (s["k"], s["ks"]), (s["v"], s["vs"]) = pool(), pool()
    if c["op"] == "append":
        s["k_new"], s["v_new"] = normal(rows, hkv, d), normal(rows, hkv, d)
        s["k_held"], s["v_held"] = torch.zeros(rows, hkv, d, dtype=t, device=dev), torch.zeros(rows, hkv, d, dtype=t, device=dev)
    else:
        s["q"] = normal(rows, hq, d, std=2.0)  # peaked softmaxes, as trained heads have
        s["lse"] = torch.zeros(rows, hq, device=dev)
        s["out"] = torch.zeros(rows, hq, d, dtype=t, device=dev)
    if own:
        from block_drafter_gb300.paged import PagedCache4
        s["cache"] = PagedCache4(s["k"], s["ks"], s["v"], s["vs"], n_q_heads=hq, dtype=t)
        s["batch"] = s["cache"].batch(table, s["n"], s["start"], n_rows=rows, max_rows=max(r), max_len=max(n))
    return s


# ------------------------------------------------------------------ plain forms
def _plan_plain(s):
    ps, dev, n_rows = s["page"], s["len"].device, s["rows"]
    n, new, held, B = s["len"].long(), s["new"].long(), s["held"].long(), s["B"]
    need = torch.div(n + new + ps - 1, ps, rounding_mode="floor")
    gains = (need - held).clamp(min=0)
    gives = (held - need).clamp(min=0) if s["give"] else torch.zeros_like(held)
    free = s["free"].long()
    # pages given back go on the stack in request and table order, then pages are taken off its top in that order
    col = torch.arange(s["table"].shape[1], device=dev)[None]
    table, stack = s["table"].clone(), s["stack"].clone()
    back = (col >= need[:, None]) & (col < held[:, None]) & (gives > 0)[:, None]
    stack[free + torch.arange(int(back.sum()), device=dev)] = table[back]
    top = free + gives.sum()
    end = gains.cumsum(0)
    served = (end <= top) | (gains == 0)
    take = (col >= held[:, None]) & (col < need[:, None]) & served[:, None]
    at = top - 1 - ((end - gains)[:, None] + col - held[:, None])
    table = torch.where(take, stack[at.clamp(min=0)], table)
    start = torch.cat((torch.zeros(1, dtype=torch.int64, device=dev), new.cumsum(0)))
    seq_len = torch.where(served, n + new, 0)
    row = torch.arange(n_rows, device=dev)
    b = (row[:, None] >= start[None, 1:]).sum(1)
    some = b < B
    bb = b.clamp(max=B - 1)
    pos = n[bb] + row - start[bb]
    some &= served[bb]
    page = table[bb, torch.div(pos, ps, rounding_mode="floor").clamp(max=table.shape[1] - 1)].long()
    keep = torch.where(served, torch.where(gives > 0, need, torch.maximum(held, need)), held)
    s["table"].copy_(table)
    s["stack"].copy_(stack)
    return (seq_len.int(), start.int(), torch.where(b < B, b, -1).int(), torch.where(some, pos, -1).int(),
            torch.where(some, page * ps + pos % ps, -1), s["table"], keep.int(), (top - (gains * served).sum()).int(), s["stack"],
            (~served).sum()[None].int())


def _heads_plain(s):
    angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin, half = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None], s["rotary"] // 2

    def one(x, gain):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.float()
        a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if s["interleaved"] else (x[..., :half], x[..., half:2 * half])
        turned = (a * cos - b * sin, a * sin + b * cos)
        turned = torch.stack(turned, -1).flatten(-2) if s["interleaved"] else torch.cat(turned, -1)
        return torch.cat((turned, x[..., 2 * half:]), -1).to(s["q"].dtype)

    return one(s["q"], s["q_gain"]), one(s["k"], s["k_gain"])


def _logprobs_plain(s):
    x = s["logits"].float() / s["temperature"]
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    l = e.sum(1, keepdim=True)
    lse = m + torch.log(l)
    entropy = (lse - (e * x).sum(1, keepdim=True) / l)[:, 0]
    out = [torch.gather(x, 1, s["tokens"].long()) - lse, entropy, lse[:, 0]]
    if s["top"]:
        ids = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices[:, :s["top"]]
        out += [ids.int(), torch.gather(x, 1, ids) - lse]
    return tuple(out)


def _row_places(s):
    """Of each row: its request and its slot."""
    row = torch.arange(s["rows"], device=s["n"].device)
    b = (row[:, None] >= s["start"][None, 1:]).sum(1)
    return b, s["n"][b] - s["start"][b + 1] + row


def _append_plain(s):
    b, p = _row_places(s)
    page, at = s["table"][b, p // s["page"]].long(), p % s["page"]
    held = []
    for x, codes, scales in ((s["k_new"], s["k"], s["ks"]), (s["v_new"], s["v"], s["vs"])):
        c, sc = _encode(x)
        codes[page, :, at] = c
        scales.view(torch.uint8)[page, :, at] = sc.view(torch.uint8)
        held.append(_decode(c, sc).to(x.dtype))
    return held[0], held[1], s["k"], s["ks"].view(torch.uint8), s["v"], s["vs"].view(torch.uint8)


def _held(s, codes, scales):
    """Every request's slots in order, [B, KV heads, slots, D] in 32 bits; slots behind the length are zero."""
    t = s["table"].long()
    x = _decode(codes[t], scales.view(torch.uint8)[t].view(scales.dtype))
    x = x.permute(0, 2, 1, 3, 4).reshape(s["B"], s["hkv"], -1, s["d"])[:, :, :s["max_len"]]
    return x * (torch.arange(s["max_len"], device=x.device)[None, :] < s["n"][:, None])[:, None, :, None]


def _attend_plain(s):
    b, p = _row_places(s)
    i = torch.arange(s["rows"], device=b.device) - s["start"][b]
    q = torch.zeros(s["B"], s["max_rows"], s["hkv"] * s["group"], s["d"], device=b.device)
    q[b, i] = s["q"].float()
    pos = torch.full((s["B"], s["max_rows"]), -1, device=b.device, dtype=torch.int64)
    pos[b, i] = p
    q = q.reshape(s["B"], s["max_rows"], s["hkv"], s["group"], s["d"]).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(s["B"], s["hkv"], -1, s["d"]), _held(s, s["k"], s["ks"]).transpose(2, 3)) * s["scale"]
    j = torch.arange(s["max_len"], device=b.device)
    seen = j <= pos[:, :, None]
    if s["window"]:
        seen = seen & ((j > pos[:, :, None] - s["window"]) | (j < s["sinks"]))
    x = x.reshape(s["B"], s["hkv"], s["group"], s["max_rows"], s["max_len"]).masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    lse = (m + torch.log(l))[..., 0].permute(0, 3, 1, 2)[b, i].reshape(s["rows"], -1)
    o = torch.matmul(x.reshape(s["B"], s["hkv"], -1, s["max_len"]), _held(s, s["v"], s["vs"])).reshape(*x.shape[:4], s["d"])
    o = torch.where(l > 0, o / l, 0.0)
    o = o.permute(0, 3, 1, 2, 4)[b, i].reshape(s["rows"], -1, s["d"])
    return o.to(s["q"].dtype), lse.contiguous()


def run(s):
    if not own:
        return {"plan": _plan_plain, "heads": _heads_plain, "logprobs": _logprobs_plain, "append": _append_plain,
                "attend": _attend_plain}[s["op"]](s)
    if s["op"] == "plan":
        s["pages"].plan(s["len"], s["new"], s["seq_len"], s["row_start"], s["pos"], s["slot"], row_request=s["request"], n_short=s["n_short"],
                        give_back=s["give"])
        return (s["seq_len"], s["row_start"], s["request"], s["pos"], s["slot"], s["table"], s["held_out"], s["free_out"], s["stack"],
                s["n_short"])
    if s["op"] == "heads":
        s["op_"](s["q"], s["k"], s["pos"], s["q_out"], s["k_out"])
        return s["q_out"], s["k_out"]
    if s["op"] == "logprobs":
        from block_drafter_gb300.target import token_logprobs
        if not s["top"]:
            token_logprobs(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"], lse=s["lse"], temperature=s["temperature"])
            return s["logprob"], s["entropy"], s["lse"]
        token_logprobs(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"], lse=s["lse"], top_ids=s["ids"], top_logprob=s["alt"],
                       temperature=s["temperature"])
        return s["logprob"], s["entropy"], s["lse"], s["ids"], s["alt"]
    if s["op"] == "append":
        s["cache"].append(s["batch"], s["k_new"], s["v_new"], k_held=s["k_held"], v_held=s["v_held"])
        return s["k_held"], s["v_held"], s["k"], s["ks"].view(torch.uint8), s["v"], s["vs"].view(torch.uint8)
    s["cache"].attention(s["batch"], s["q"], s["out"], lse=s["lse"], window=s["window"], n_sink=s["sinks"])
    return s["out"], s["lse"]


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    return {"plan": _plan_exact, "heads": _heads_exact, "logprobs": _logprobs_exact, "append": _append_exact, "attend": _attend_exact}[c["op"]](c, s)


def _plan_exact(c, s):
    """Request by request, as the step would be planned on the host."""
    n, r, held, width, need = _pages(c)
    ps, rows = c["page"], s["rows"]
    table, stack, free = s["table"].cpu().numpy().copy(), s["stack"].cpu().numpy().copy(), int(s["free"])
    keep, promised, short = list(held), 0, 0
    for b in range(c["B"]):
        if c["give"] and need[b] < held[b]:
            stack[free:free + held[b] - need[b]] = table[b, need[b]:held[b]]
            free, keep[b] = free + held[b] - need[b], need[b]
    top = free
    seq, pos, slot, req = [], np.full(rows, -1, np.int32), np.full(rows, -1, np.int64), np.full(rows, -1, np.int32)
    start = [0]
    for b in range(c["B"]):
        first, start = start[-1], start + [start[-1] + r[b]]
        req[first:first + r[b]] = b
        more = max(0, need[b] - held[b])
        promised += more
        if more and promised > top:
            short += 1
            seq.append(0)
            continue
        for x in range(more):
            free -= 1
            table[b, held[b] + x] = stack[free]
        keep[b] = max(keep[b], need[b])
        seq.append(n[b] + r[b])
        j = np.arange(n[b], n[b] + r[b])
        pos[first:first + r[b]] = j
        slot[first:first + r[b]] = table[b, j // ps].astype(np.int64) * ps + j % ps
    i = lambda x: np.array(x, dtype=np.int32)  # noqa: E731
    return i(seq), i(start), req, pos, slot, table, i(keep), i([free]), stack, i([short])


def _heads_exact(c, s):
    half = c["rotary"] // 2
    z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["pos"].double()[:, None] * s["freq"][None])[:, None]
    out = []
    for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
        y = x.double() / torch.sqrt(x.double().pow(2).mean(-1, keepdim=True) + EPS) * gain.double()
        if c["interleaved"]:
            w = torch.view_as_complex(y[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * z
            y[..., :2 * half] = torch.view_as_real(w).flatten(-2)
        else:
            w = torch.complex(y[..., :half], y[..., half:2 * half]) * z
            y[..., :half], y[..., half:2 * half] = w.real, w.imag
        out.append(y)
    return tuple(out)


def _logprobs_exact(c, s):
    parts = []
    for i in range(0, c["rows"], 64):  # 64 rows at a time
        raw = s["logits"][i:i + 64].double()
        z = raw / c["temperature"]
        lp = z - torch.logsumexp(z, 1, keepdim=True)
        one = [torch.gather(lp, 1, s["tokens"][i:i + 64].long()), -(lp.exp() * lp).sum(1), torch.logsumexp(z, 1)]
        if c["top"]:
            v, ids = raw.clone(), []
            for _ in range(c["top"]):  # the largest, the first of equals
                m = v.amax(1, keepdim=True)
                k = (v == m).to(torch.uint8).argmax(1, keepdim=True)
                ids.append(k)
                v.scatter_(1, k, -math.inf)
            ids = torch.cat(ids, 1)
            one += [ids.int(), torch.gather(lp, 1, ids)]
        parts.append(one)
    return tuple(torch.cat(x) for x in zip(*parts))


def _nearest(x):
    """_encode by search: the scale nearest to the largest magnitude / 6 among all e4m3 numbers, the codes nearest to
    the values among all e2m1 ones; of two as near the one with the even code.  [..., D] in numpy, 64 bits."""
    x = x.reshape(*x.shape[:-1], -1, 16)
    byte = np.arange(127)
    e, f = byte >> 3, byte & 7
    e4m3 = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e - 7.0))

    def pick(table, v):
        hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
        lo = hi - 1
        down, up = v - table[lo], table[hi] - v
        return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)

    # compared as 6 s with the magnitude and as s g with the values: products of few bits, exact in 64
    scale = pick(6 * e4m3, np.abs(x).max(-1))
    s = e4m3[scale][..., None]
    grid = np.array(GRID)
    code = np.zeros(x.shape, dtype=np.uint8)
    for i in range(1, 8):  # past the middle between codes i - 1 and i, or on it where i is even
        mid = s * (grid[i - 1] + grid[i]) / 2
        code += (np.abs(x) > mid) | ((np.abs(x) == mid) & (i % 2 == 0))
    code = np.where(s > 0, code | (np.signbit(x).astype(np.uint8) << 3), 0).astype(np.uint8)
    val = np.where(code & 8, -1.0, 1.0) * grid[code & 7] * s
    code = code.reshape(*code.shape[:-2], -1)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.astype(np.uint8), val.reshape(*val.shape[:-2], -1)


def _append_exact(c, s):
    n, r = _lengths(c)
    if sum(r) * c["hkv"] * c["d"] > 1 << 24:
        return None
    first, ps, out, held = [0] + list(np.cumsum(r)), c["page"], [], []
    for x, codes, scales in ((s["k_new"], s["k"], s["ks"]), (s["v_new"], s["v"], s["vs"])):
        code, scale, val = _nearest(x.double().cpu().numpy())
        codes, scales = codes.clone(), scales.view(torch.uint8).clone()
        for b in range(c["B"]):
            slot = torch.arange(n[b] - r[b], n[b], device="cuda")
            page = s["table"][b].long()[torch.div(slot, ps, rounding_mode="floor")]
            rows = slice(first[b], first[b + 1])
            codes.permute(0, 2, 1, 3)[page, slot % ps] = torch.from_numpy(code[rows]).cuda()
            scales.permute(0, 2, 1, 3)[page, slot % ps] = torch.from_numpy(scale[rows]).cuda()
        held.append(val)
        out += [codes, scales]
    return held[0], held[1], out[0], out[1], out[2], out[3]


def _attend_exact(c, s):
    """Request by request, KV head by KV head, over each request's own slots alone."""
    n, r = _lengths(c)
    ps, d, group, hkv = c["page"], c["d"], c["group"], c["hkv"]
    if sum(a * b for a, b in zip(n, r)) * hkv * group > 1 << 32:
        return None
    first = [0] + list(np.cumsum(r))
    out = torch.zeros(sum(r), hkv * group, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(r), hkv * group, dtype=torch.float64, device="cuda")
    values = torch.tensor([[g if i < 8 else -g for g in (GRID + GRID)[i:i + 1]][0] for i in range(16)], dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        j = torch.arange(n[b], device="cuda")
        page, off = s["table"][b].long()[j // ps], j % ps
        at = (n[b] - r[b] + torch.arange(r[b], device="cuda"))[:, None]
        hidden = j[None] > at
        if c["window"]:
            hidden |= (at - j[None] >= c["window"]) & (j[None] >= c["sinks"])
        for h in range(hkv):
            k, v = (torch.stack((values[(x[page, h, off] & 15).long()], values[(x[page, h, off] >> 4).long()]), 2).reshape(n[b], d)
                    * sc.view(torch.uint8)[page, h, off].view(sc.dtype).double().repeat_interleave(16, 1)
                    for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])))
            rows = slice(first[b], first[b + 1])
            for e in range(group):
                z = (s["q"][rows, h * group + e].double() @ k.T) / math.sqrt(d)
                z = z.masked_fill(hidden, -math.inf)
                lse[rows, h * group + e] = torch.logsumexp(z, 1)
                out[rows, h * group + e] = torch.softmax(z, 1) @ v
    return out, lse
