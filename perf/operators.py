"""Measured cases of the paged-cache operators: append, attention (decode, verification,
prompt chunks; sliding window and sinks), accumulated attention weights, eviction.

The pool is [pages, KV heads, page size, head dim]; request b holds seq_len[b] slots in the
pages that row b of the page table names, and its new rows are the last ones of them.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def _case(op, *, name=None, dtype="bf16", B, hkv=8, group=4, d=128, page=64, lo, hi, rlo, rhi, window=0, sinks=0,
          used=0, budget=0, recent=0, lens=1):
    """lo..hi: slots held by a request; rlo..rhi: its new rows; used: rows whose weights count
    (0: all); lens: what the lengths are drawn from."""
    c = dict(op=op, dtype=dtype, B=B, hkv=hkv, group=group, d=d, page=page, lo=lo, hi=hi, rlo=rlo, rhi=rhi, window=window,
             sinks=sinks, used=used, budget=budget, recent=recent, lens=lens)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the rows of eight verified blocks go into the target's cache (concurrency 8, 16-row blocks)
        _case("append", name="append_block_b8", B=8, lo=512, hi=16384, rlo=16, rhi=16),
        # ragged prompt chunks of four requests, small pages
        _case("append", name="append_chunk_b4", dtype="fp16", B=4, page=16, lo=8192, hi=9001, rlo=2048, rhi=8191, lens=2),
        # one new token of one request at the 27B geometry's context
        _case("attention", name="decode_b1_4096", B=1, lo=4096, hi=4096, rlo=1, rhi=1),
        # one new token for each of sixteen long, ragged contexts
        _case("attention", name="decode_b16_long", dtype="fp16", B=16, page=16, lo=4096, hi=32768, rlo=1, rhi=1, lens=3),
        # one new token through a sliding-window layer with four sink tokens
        _case("attention", name="decode_b8_window", B=8, page=32, lo=4096, hi=32768, rlo=1, rhi=1, window=4096, sinks=4, lens=4),
        # a drafted block of sixteen rows is verified for eight requests
        _case("attention", name="verify_b8_w16", B=8, lo=512, hi=16384, rlo=16, rhi=16, lens=5),
        # ragged prompt chunks through a sliding-window layer with sinks, small heads, odd lengths
        _case("attention", name="chunk_b3_window", dtype="fp16", B=3, hkv=2, group=2, d=64, page=16, lo=2049, hi=6001, rlo=517, rhi=2047,
              window=1024, sinks=4, lens=6),
        # a whole prompt of 8192 tokens, full attention
        _case("attention", name="prompt_8192", B=1, lo=8192, hi=8192, rlo=8192, rhi=8192),
        # accumulated weights of one decoded token each
        _case("weights", name="weights_b8_token", B=8, lo=512, hi=16384, rlo=1, rhi=1, lens=7),
        # accumulated weights of the last 64 rows of a prompt, through a window with sinks
        _case("weights", name="weights_b2_prompt", dtype="fp16", B=2, page=32, lo=6000, hi=16383, rlo=64, rhi=64, window=4096, sinks=4, lens=8),
        # one request's cache goes from 4096 slots to 2048
        _case("evict", name="evict_b1_4096", B=1, lo=4096, hi=4096, rlo=0, rhi=0, budget=2048, sinks=4, recent=256),
        # eight ragged caches go to 8192 slots at most
        _case("evict", name="evict_b8_long", dtype="fp16", B=8, page=16, lo=4096, hi=32768, rlo=0, rhi=0, budget=8191, sinks=4, recent=512, lens=9),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    """One case of the same ranges: lengths 1 to 32768, blocks of 1 to 16 rows or prompt chunks
    of up to 8192, one to eight KV heads, groups of one to eight, pages of 8 to 256 slots (odd ones
    too), with and without a window."""
    heads = dict(hkv=rng.choice([1, 2, 4, 8]), group=rng.choice([1, 2, 3, 4, 5, 8]), d=rng.choice([64, 128, 128]),
                 dtype=rng.choice(["bf16", "fp16"]), page=rng.choice([8, 16, 24, 32, 33, 64, 128, 256]), lens=rng.randrange(10, 1 << 20))
    op = rng.choice(["append", "attention", "attention", "attention", "weights", "evict"])
    win = dict(window=_log(rng, 16, 8192), sinks=rng.choice([0, 1, 4, 17, 128])) if rng.random() < 0.4 else {}
    B = rng.choice([1, 1, 2, 3, 4, 5, 8, 12, 16])
    hi = _log(rng, 1, 32768)
    lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
    if op == "append":
        rhi = min(hi, _log(rng, 1, 8192))
        B = max(1, min(B, 65536 // hi))
        return _case(op, B=B, lo=max(lo, rhi), hi=hi, rlo=max(1, int(rhi * rng.uniform(0.2, 1.0))), rhi=rhi, **heads)
    if op == "evict":
        budget = max(1, int(hi * rng.uniform(0.2, 1.1)))
        sinks = min(rng.choice([0, 1, 4, 64]), budget)
        kept = min(hi, budget) * heads["hkv"] * heads["d"]  # no more moves than the largest listed case has
        return _case(op, B=max(1, min(B, (1 << 26) // kept)), lo=lo, hi=hi, rlo=0, rhi=0, budget=budget, sinks=sinks,
                     recent=int((budget - sinks) * rng.uniform(0, 0.5)), **heads)
    if op == "attention" and rng.random() < 0.4:  # prompt chunks; no more score entries than the largest listed case has
        rhi = min(hi, _log(rng, 17, 8192))
        B = max(1, min(B, (1 << 30) // (heads["hkv"] * heads["group"] * hi * rhi), 65536 // hi))
    else:  # tokens and blocks
        rhi = min(hi, rng.choice([1, 1, 2, 3, 5, 7, 8, 13, 16]))
    c = _case(op, B=B, lo=max(lo, rhi), hi=hi, rlo=max(1, rhi - rng.randrange(0, 1 + rhi // 2)), rhi=rhi, **heads, **win)
    if op == "weights":
        c["used"] = rng.choice([0, 1 + rng.randrange(rhi)])
    return c


def _lengths(c):
    r = random.Random(c["lens"])
    n = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    return n, [r.randint(min(c["rlo"], x), min(c["rhi"], x)) for x in n]


def _pairs(n, r, window, sinks, used):
    """(slots visible to some row, visible pairs) of the first `used` of r rows at the end of n slots."""
    if not used:
        return 0, 0
    p = np.arange(n - r, n - r + used, dtype=np.int64)
    if not window:
        return int(p[-1]) + 1, int((p + 1).sum())
    first = np.maximum(0, p - window + 1)
    seen = int(p[-1]) + 1 - int(first[0]) + min(sinks, int(first[0]))
    return seen, int((p + 1 - first + np.minimum(sinks, first)).sum())


def work(c):
    n, r = _lengths(c)
    hq, hkv, d, e = c["hkv"] * c["group"], c["hkv"], c["d"], 2
    rows = sum(r)
    kv = hkv * d * e  # one slot's keys
    table = 4 * sum(-(-x // c["page"]) for x in n)
    if c["op"] == "append":
        return {"bytes": 4 * rows * kv + 4 * rows, "flops": 0}
    if c["op"] == "evict":
        kept = sum(min(x, c["budget"]) for x in n)
        return {"bytes": 4 * sum(n) + 4 * kept * kv + 8 * kept + table, "flops": 0}
    used = [min(x, c["used"]) if c["op"] == "weights" and c["used"] else x for x in r]
    seen, pairs = (sum(v) for v in zip(*(_pairs(a, b, c["window"], c["sinks"], u) for a, b, u in zip(n, r, used))))
    if c["op"] == "weights":
        return {"bytes": seen * kv + sum(used) * hq * (d * e + 4) + 8 * sum(n) + table, "flops": 2 * d * hq * pairs}
    return {"bytes": 2 * seen * kv + rows * hq * (2 * d * e + 4) + table, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs
def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, dev = TYPES[c["dtype"]], "cuda"
    n, r = _lengths(c)
    B, hkv, hq, d, ps = c["B"], c["hkv"], c["hkv"] * c["group"], c["d"], c["page"]
    held = [-(-x // ps) for x in n]
    dest = [-(-min(x, c["budget"]) // ps) for x in n]  # pages that an eviction fills
    cols, dcols, total = max(held), max(dest), sum(held) + sum(dest)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std).to(t)

    ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)  # pages lie anywhere in the pool
    table = torch.zeros(B, cols, dtype=torch.int32, device=dev)
    dst = torch.zeros(B, max(1, dcols), dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
        dst[b, :dest[b]] = ids[at:at + dest[b]]
        at += dest[b]
    s = dict(c, total=total, cols=cols, n=torch.tensor(n, dtype=torch.int32, device=dev), max_len=max(n), max_rows=max(r),
             start=torch.tensor([0] + list(np.cumsum(r)), dtype=torch.int32, device=dev), table=table, dst=dst, rows=sum(r),
             k=normal(total, hkv, ps, d), v=normal(total, hkv, ps, d), scale=1.0 / math.sqrt(d))
    if c["op"] == "append":
        s["k_new"], s["v_new"] = normal(sum(r), hkv, d), normal(sum(r), hkv, d)
    elif c["op"] == "evict":
        # accumulated weights are spread over decades
        s["score"] = torch.exp(2.0 * torch.randn(B, max(n), generator=g, device=dev))
        s["score_out"] = torch.zeros(B, c["budget"], device=dev)
        s["kept"] = torch.full((B, c["budget"]), -1, dtype=torch.int32, device=dev)
        s["len_out"] = torch.zeros(B, dtype=torch.int32, device=dev)
    else:
        s["q"] = normal(sum(r), hq, d, std=2.0)  # peaked softmaxes, as trained heads have
        s["lse"] = torch.zeros(sum(r), hq, device=dev)
        if c["op"] == "attention":
            s["out"] = torch.zeros(sum(r), hq, d, dtype=t, device=dev)
        else:
            s["used"] = torch.tensor([min(x, c["used"]) if c["used"] else x for x in r], dtype=torch.int32, device=dev)
            s["score"] = torch.exp(torch.randn(B, max(n), generator=g, device=dev))
            s["score_out"] = torch.zeros(B, max(n), device=dev)
            s["lse"] = _attention(s, False)[1]  # the attention before it wrote them
    if own:
        from block_drafter_gb300.paged import PagedCache
        s["cache"] = PagedCache(s["k"], s["v"], n_q_heads=hq)
        s["batch"] = s["cache"].batch(table, s["n"], s["start"], n_rows=sum(r), max_rows=max(r), max_len=max(n))
    return s


# ------------------------------------------------------------------ plain forms
def _held(s, pool):
    """Every request's slots in order, [B, KV heads, slots, D] in 32 bits; slots behind the length are zero."""
    x = pool[s["table"].long()].permute(0, 2, 1, 3, 4).reshape(s["B"], s["hkv"], -1, s["d"])[:, :, :s["max_len"]].float()
    slot = torch.arange(s["max_len"], device=x.device)
    return x * (slot[None, :] < s["n"][:, None])[:, None, :, None]


def _row_places(s):
    """Of each row: its request and its slot."""
    row = torch.arange(s["rows"], device=s["n"].device)
    b = (row[:, None] >= s["start"][None, 1:]).sum(1)
    return b, s["n"][b] - s["start"][b + 1] + row


def _scores(s):
    """Scaled scores [B, KV heads, group, rows, slots], -inf where a slot is not visible."""
    b, p = _row_places(s)
    i = torch.arange(s["rows"], device=b.device) - s["start"][b]
    q = torch.zeros(s["B"], s["max_rows"], s["hkv"] * s["group"], s["d"], device=b.device)
    q[b, i] = s["q"].float()
    pos = torch.full((s["B"], s["max_rows"]), -1, device=b.device, dtype=torch.int64)
    pos[b, i] = p
    q = q.reshape(s["B"], s["max_rows"], s["hkv"], s["group"], s["d"]).permute(0, 2, 3, 1, 4)
    k = _held(s, s["k"])
    x = torch.matmul(q.reshape(s["B"], s["hkv"], -1, s["d"]), k.transpose(2, 3)) * s["scale"]
    j = torch.arange(s["max_len"], device=b.device)
    seen = j <= pos[:, :, None]
    if s["window"]:
        seen = seen & ((j > pos[:, :, None] - s["window"]) | (j < s["sinks"]))
    x = x.reshape(s["B"], s["hkv"], s["group"], s["max_rows"], s["max_len"])
    return x.masked_fill_(~seen[:, None, None], -math.inf), b, i


def _attention(s, values=True):
    x, b, i = _scores(s)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    lse = (m + torch.log(l))[..., 0].permute(0, 3, 1, 2)[b, i].reshape(s["rows"], -1)
    if not values:
        return None, lse.contiguous()
    v = _held(s, s["v"])
    o = torch.matmul(x.reshape(s["B"], s["hkv"], -1, s["max_len"]), v).reshape(*x.shape[:4], s["d"])
    o = torch.where(l > 0, o / l, 0.0)
    o = o.permute(0, 3, 1, 2, 4)[b, i].reshape(s["rows"], -1, s["d"])
    return o.to(s["q"].dtype), lse.contiguous()


def _weights(s):
    x, b, i = _scores(s)
    counts = torch.arange(s["max_rows"], device=b.device) < s["used"][:, None]
    lse = torch.zeros(s["B"], s["max_rows"], s["hkv"] * s["group"], device=b.device)
    lse[b, i] = s["lse"]
    lse = lse.reshape(s["B"], s["max_rows"], s["hkv"], s["group"]).permute(0, 2, 3, 1)
    w = x.sub_(lse[..., None]).exp_().masked_fill_(~counts[:, None, None, :, None], 0.0).sum((1, 2, 3))
    held = torch.arange(s["max_len"], device=b.device) < s["n"][:, None]
    return torch.where(held, DECAY * s["score"] + w, s["score_out"])


def _evict(s):
    n, budget = s["n"][:, None].long(), s["budget"]
    j = torch.arange(s["max_len"], device=n.device)[None, :]
    key = s["score"].masked_fill((j < s["sinks"]) | (j >= n - s["recent"]), math.inf).masked_fill(j >= n, -math.inf)
    rank = torch.sort(key, dim=1, descending=True, stable=True).indices
    keep = torch.zeros_like(key, dtype=torch.bool).scatter_(1, rank[:, :budget], True) & (j < n)
    new = keep.long().cumsum(1) - 1
    b, old = keep.nonzero(as_tuple=True)
    new = new[b, old]
    ps = s["page"]
    src, dst = s["table"][b, old // ps].long(), s["dst"][b, new // ps].long()
    for pool in (s["k"], s["v"]):
        pool[dst, :, new % ps] = pool[src, :, old % ps]
    kept, score = s["kept"].clone(), s["score_out"].clone()
    kept[b, new] = old.int()
    score[b, new] = s["score"][b, old]
    return kept, keep.sum(1).int(), score


DECAY = 0.9375


def run(s):
    if own:
        cache, batch = s["cache"], s["batch"]
        if s["op"] == "append":
            cache.append(batch, s["k_new"], s["v_new"])
            return s["k"], s["v"]
        if s["op"] == "attention":
            cache.attention(batch, s["q"], s["out"], lse=s["lse"], window=s["window"], n_sink=s["sinks"])
            return s["out"], s["lse"]
        if s["op"] == "weights":
            cache.weights(batch, s["q"], s["lse"], s["score_out"], score_in=s["score"], decay=DECAY, rows_used=s["used"],
                          window=s["window"], n_sink=s["sinks"])
            return s["score_out"]
        cache.evict(batch, s["score"], s["budget"], s["kept"], s["len_out"], n_sink=s["sinks"], n_recent=s["recent"],
                    dst_table=s["dst"], score_out=s["score_out"])
        return s["kept"], s["len_out"], s["score_out"], s["k"], s["v"]
    if s["op"] == "append":
        b, p = _row_places(s)
        page = s["table"][b, p // s["page"]].long()
        s["k"][page, :, p % s["page"]] = s["k_new"]
        s["v"][page, :, p % s["page"]] = s["v_new"]
        return s["k"], s["v"]
    if s["op"] == "attention":
        return _attention(s)
    if s["op"] == "weights":
        return _weights(s)
    return _evict(s) + (s["k"], s["v"])


# ------------------------------------------------------------------ the definition in 64 bits
def exact(c, seed):
    """Request by request, KV head by KV head, over each request's own slots alone."""
    s = prepare(c, seed)
    n, r = _lengths(c)
    ps, d, group, hkv = c["page"], c["d"], c["group"], c["hkv"]
    first = [0] + list(np.cumsum(r))
    if c["op"] == "append":
        k, v = s["k"].clone(), s["v"].clone()
        for b in range(c["B"]):
            slot = torch.arange(n[b] - r[b], n[b], device="cuda")
            page = s["table"][b].long()[torch.div(slot, ps, rounding_mode="floor")]
            for pool, new in ((k, s["k_new"]), (v, s["v_new"])):
                pool.permute(0, 2, 1, 3)[page, slot - slot // ps * ps] = new[first[b]:first[b + 1]]
        return k, v
    if c["op"] == "evict":
        kept = s["kept"].cpu().numpy().copy()
        score = s["score_out"].cpu().numpy().copy()
        k, v = s["k"].clone(), s["v"].clone()
        old = s["score"].cpu().numpy()
        length = []
        for b in range(c["B"]):
            if n[b] <= c["budget"]:
                ids = np.arange(n[b])
            else:
                a, z = c["sinks"], n[b] - c["recent"]
                best = np.argsort(-old[b, a:z].astype(np.float64), kind="stable")[:c["budget"] - a - c["recent"]] + a
                ids = np.sort(np.concatenate([np.arange(a), best, np.arange(z, n[b])]))
            m = len(ids)
            length.append(m)
            kept[b, :m], score[b, :m] = ids, old[b, ids]
            o, w = torch.from_numpy(ids).cuda(), torch.arange(m, device="cuda")
            for pool, was in ((k, s["k"]), (v, s["v"])):
                rows = was.permute(0, 2, 1, 3)[s["table"][b].long()[o // ps], o % ps]
                pool.permute(0, 2, 1, 3)[s["dst"][b].long()[w // ps], w % ps] = rows
        return kept, np.array(length, dtype=np.int32), score.astype(np.float64), k, v
    if sum(a * b for a, b in zip(n, r)) * hkv * group > 1 << 32:
        return None
    out = torch.zeros(sum(r), hkv * group, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(r), hkv * group, dtype=torch.float64, device="cuda")
    score = s["score_out"].double() if c["op"] == "weights" else None
    for b in range(c["B"]):
        j = torch.arange(n[b], device="cuda")
        page, off = s["table"][b].long()[j // ps], j % ps
        used = int(s["used"][b]) if score is not None else r[b]
        if score is not None:
            score[b, :n[b]] = DECAY * s["score"][b, :n[b]].double()
        at = (n[b] - r[b] + torch.arange(used, device="cuda"))[:, None]
        hidden = j[None] > at
        if c["window"]:
            hidden |= (at - j[None] >= c["window"]) & (j[None] >= c["sinks"])
        for h in range(hkv):
            k, rows, heads = s["k"][page, h, off].double(), slice(first[b], first[b] + used), slice(h * group, (h + 1) * group)
            for e in range(group):
                z = (s["q"][rows, h * group + e].double() @ k.T) / math.sqrt(d)
                if score is not None:
                    score[b, :n[b]] += torch.exp(z - s["lse"][rows, h * group + e, None].double()).masked_fill(hidden, 0).sum(0)
                    continue
                z = z.masked_fill(hidden, -math.inf)
                lse[rows, h * group + e] = torch.logsumexp(z, 1)
                out[rows, h * group + e] = torch.softmax(z, 1) @ s["v"][page, h, off].double()
    return score if score is not None else (out, lse)
