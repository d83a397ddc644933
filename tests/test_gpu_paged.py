"""Paged cache on the GPU against the fp64 oracle: append, attention, accumulated weights,
eviction, and a run of them together.  Every place no request holds is NaN in the pools."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from paged_harness import TYPES, PagedCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from block_drafter_gb300 import builder
    builder.build()


def sync():
    from block_drafter_gb300 import binding
    binding.sync_status()


# ------------------------------------------------------------------ attention
ATTENTION = {
    "one_slot": PagedCase((1,), (1,)),
    "one_token_each": PagedCase((1, 2, 15, 16, 17, 63, 64, 65), (1,) * 8),
    "ragged": PagedCase((5, 130, 700, 257, 1), (1, 3, 2, 1, 1), lead=2),
    "fp16_d64": PagedCase((33, 400, 1000), (1, 1, 1), d=64, dtype="fp16", group=1, hkv=3),
    "long": PagedCase((5000, 4097), (1, 1), hkv=1, group=8),
    "wide_group": PagedCase((300, 77), (1, 2), hkv=1, group=32),
    "widest_group": PagedCase((200, 40), (2, 1), hkv=1, group=128, d=64),
    "odd_group": PagedCase((100, 321), (3, 5), group=5, hkv=2),
    "block": PagedCase((600, 16, 1111), (16, 16, 16)),
    "block_window": PagedCase((600, 40, 1111), (16, 7, 13), window=64, n_sink=4),
    "window_token": PagedCase((600, 40, 1111, 3), (1, 1, 1, 1), window=100, n_sink=3),
    "window_no_sinks": PagedCase((601, 40), (1, 2), window=17),
    "window_one": PagedCase((300, 20), (2, 1), window=1),
    "window_one_sink": PagedCase((300, 20), (2, 18), window=1, n_sink=1),
    "sinks_reach_window": PagedCase((90, 300), (4, 4), window=50, n_sink=60),
    "sinks_beyond_length": PagedCase((50, 300), (4, 40), window=8, n_sink=1000),
    "window_beyond_length": PagedCase((50, 130), (4, 40), window=5000, n_sink=2),
    "page_1": PagedCase((37, 129), (1, 9), page=1),
    "page_odd": PagedCase((37, 200, 66), (1, 9, 33), page=33),
    "page_256": PagedCase((300, 257), (1, 40), page=256),
    "nhd_pool": PagedCase((137, 256), (1, 20), nhd=True),
    "padded": PagedCase((137, 250), (1, 20), pad=8, lead=3),
    "nhd_padded_fp16": PagedCase((137, 250), (30, 20), pad=8, nhd=True, dtype="fp16", d=64),
    "chunk": PagedCase((300, 64), (130, 64)),
    "chunk_whole": PagedCase((333,), (333,), hkv=1),
    "chunk_mha": PagedCase((333, 129), (200, 129), hkv=3, group=1),
    "chunk_fp16_d64": PagedCase((400, 255), (257, 255), d=64, dtype="fp16", lead=5),
    "chunk_window": PagedCase((700, 300), (300, 130), window=128, n_sink=4),
    "chunk_window_odd": PagedCase((701, 299), (301, 299), window=77, n_sink=130, group=3),
    "chunk_and_tokens": PagedCase((500, 20, 1, 900, 40), (200, 1, 1, 1, 39)),
    "more_rows_than_slots": PagedCase((5, 0, 100), (9, 3, 120), lead=1),
    "empty_requests": PagedCase((0, 50, 20, 0), (0, 0, 2, 1)),
    "peaked": PagedCase((400, 130), (1, 60), std=12.0),
    "peaked_fp16": PagedCase((400, 130), (1, 60), std=12.0, dtype="fp16"),
    "table_has_spare_entries": PagedCase((40, 90), (1, 50), spare=5),
}


@pytest.mark.parametrize("name", list(ATTENTION))
def test_attention_matches_the_oracle(name):
    c = ATTENTION[name].build()
    out, lse = c.attend()
    sync()
    c.check_attention(out, lse)
    c.check_guards(out, lse)
    again, lse2 = c.attend()
    assert torch.equal(out, again) and torch.equal(lse, lse2)   # nothing depends on the run


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128])
@pytest.mark.parametrize("d,group", [(128, 4), (64, 1)])
def test_attention_of_every_row_count(rows, d, group):
    c = PagedCase((rows + 150, 129 + rows), (rows, rows), d=d, group=group, hkv=1, seed=rows).build()
    out, lse = c.attend()
    sync()
    c.check_attention(out, lse)


def test_attention_without_lse_and_with_a_scale():
    c = PagedCase((90, 200), (1, 40)).build()
    c.scale = 0.3
    out, lse = c.attend(scale=0.3)
    c.check_attention(out, lse)
    alone, _ = c.outputs()
    c.cache.attention(c.batch, c.qd, alone, scale=0.3)
    sync()
    assert torch.equal(alone, out)


@pytest.mark.parametrize("rows,window", [(1, 0), (4, 0), (4, 20), (100, 0), (100, 40)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_garbage_in_slots_a_row_does_not_see_stays_out(rows, window, bad):
    """Slots of later rows, and slots the window hides from later rows, hold infinities or NaN:
    only the rows that see them may show it."""
    c = PagedCase((260, 300), (rows, rows), window=window, n_sink=2, hkv=1).build()
    hit = [c.lens[0] - 1]                       # the last row's own slot: earlier rows do not see it
    if window:
        hit.append(c.lens[0] - rows - window + 1)   # seen by the first row alone
    for j in hit:
        page = c.table[0, j // c.page].item()
        c.vd[page, 0, j % c.page, 3] = bad
    out, lse = c.attend()
    sync()
    got = out[:rows].double().cpu().numpy()
    see = P.visible(c.lens[0], rows, window, 2)
    for i in range(rows):
        touched = any(see[i, j] for j in hit)
        fine = np.ones((c.group, c.d), bool)
        fine[:, 3] = not touched
        assert (np.isfinite(got[i]) == fine).all(), i
    clean = PagedCase((260, 300), (rows, rows), window=window, n_sink=2, hkv=1).build()
    ref, lref = clean.attend()
    keep = torch.ones_like(ref, dtype=torch.bool)
    keep[:rows, :, 3] = torch.tensor([[not any(see[i, j] for j in hit)] for i in range(rows)], device="cuda")
    torch.testing.assert_close(out[keep].float(), ref[keep].float(), rtol=2 ** -6, atol=2 ** -7)
    assert torch.equal(lse, lref)


def test_bad_keys_in_unseen_slots_stay_out():
    c = PagedCase((200,), (3,), hkv=1).build()
    c.kd[c.table[0, 199 // 16].item(), 0, 199 % 16] = float("nan")
    out, lse = c.attend()
    sync()
    assert torch.isfinite(out[:2]).all() and torch.isfinite(lse[:2]).all() and torch.isnan(out[2]).all()


def test_bad_sizes_and_pages_are_reported_and_other_requests_stand():
    from block_drafter_gb300 import binding as B
    for spoil in ("page", "negative_page", "length", "negative_length", "rows", "rows_out"):
        c = PagedCase((200, 100, 70), (2, 3, 1)).build()
        if spoil == "page":
            c.table[1, 6] = 10 ** 6                             # slots 96 .. 99
        elif spoil == "negative_page":
            c.table[1, 6] = -1
        elif spoil == "length":
            c.lend[1] = 201
        elif spoil == "negative_length":
            c.lend[1] = -5
        elif spoil == "rows":
            c.startd.copy_(torch.tensor([0, 4, 2, 6]))         # request 1 ends before it begins
        else:
            c.startd.copy_(torch.tensor([0, 2, 5, 600]))       # request 2 goes beyond the rows
        out, lse = c.attend()
        with pytest.raises(B.BdError) as err:
            B.sync_status()
        assert err.value.status == -1
        B.sync_status()
        if spoil not in ("rows", "rows_out"):
            c.check_attention(out, lse, requests=(0, 2))
        elif spoil == "rows_out":
            c.check_attention(out, lse, requests=(0, 1))
        k = torch.randn(c.n_rows, c.hkv, c.d, device="cuda").to(torch.bfloat16)
        before = c.kd.clone()
        c.cache.append(c.batch, k, k)
        with pytest.raises(B.BdError):
            B.sync_status()
        changed = (c.kd.view(torch.int16) != before.view(torch.int16)).flatten(2).any(2).any(1).sum().item()
        assert changed <= 5


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("case", [PagedCase((1,), (1,)), PagedCase((17, 300, 64), (1, 16, 64), lead=2),
                                  PagedCase((5, 0, 9), (9, 2, 0), page=4),
                                  PagedCase((700, 33), (700, 33), page=33, dtype="fp16", d=64, pad=8, nhd=True),
                                  PagedCase((3000,), (2900,), hkv=8, page=64)])
def test_append_stores_the_rows_and_nothing_else(case):
    c = case.build()
    g = torch.Generator().manual_seed(5)
    new = [torch.randn(c.n_rows, c.hkv, c.d, generator=g).to(TYPES[c.dtype]) for _ in range(2)]
    want = [c.kd.cpu().clone(), c.vd.cpu().clone()]
    for b, (n, r) in enumerate(zip(c.lens, c.rows)):
        for i in range(r):
            p = n - r + i
            if p >= 0:
                for w, x in zip(want, new):
                    w[c.table[b, p // c.page].item(), :, p % c.page] = x[c.starts[b] + i]
    c.cache.append(c.batch, c.strided(new[0]), c.strided(new[1]))
    sync()
    for got, w in zip((c.kd, c.vd), want):
        assert torch.equal(got.cpu().contiguous().view(torch.int16), w.contiguous().view(torch.int16))


# ------------------------------------------------------------------ weights
WEIGHTS = {
    "token": (PagedCase((1, 40, 700), (1, 1, 1)), None),
    "block_accepted": (PagedCase((60, 300, 90), (16, 16, 16), lead=1), (16, 3, 0)),
    "accepted_out_of_range": (PagedCase((60, 300), (5, 6)), (-3, 99)),
    "window": (PagedCase((400, 90), (9, 40), window=50, n_sink=3), None),
    "prompt": (PagedCase((300, 129), (200, 129), d=64, dtype="fp16", hkv=3, group=2), None),
    "more_rows_than_slots": (PagedCase((5, 20), (9, 1)), None),
    "wide_group": (PagedCase((200,), (3,), hkv=1, group=40), None),
    "odd_pages": (PagedCase((100, 77), (2, 5), page=7, nhd=True, pad=8), None),
    "peaked": (PagedCase((333,), (33,), std=8.0), None),
}


@pytest.mark.parametrize("inout", [False, True])
@pytest.mark.parametrize("name", list(WEIGHTS))
def test_weights_match_the_oracle(name, inout):
    case, used = WEIGHTS[name]
    c = case.build()
    _, lse = c.attend()
    B, width = len(c.lens), c.max_len + 3
    g = torch.Generator().manual_seed(3)
    start = torch.rand(B, width, generator=g).cuda()
    score = start.clone() if inout else torch.full((B, width), -7.0, device="cuda")
    ud = None if used is None else torch.tensor(used, dtype=torch.int32, device="cuda")
    kw = dict(rows_used=ud, window=c.window, n_sink=c.n_sink)
    c.cache.weights(c.batch, c.qd, lse, score, score_in=score if inout else None, decay=0.75, **kw)
    sync()
    got, lse = score.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, (n, r) in enumerate(zip(c.lens, c.rows)):
        s = slice(c.starts[b], c.starts[b] + r)
        w = P.weights(c.qf[s], c.k[b], lse[s], r if used is None else used[b], c.window, c.n_sink, c.scale)
        _, _, _, size = P.attention(c.qf[s], c.k[b], c.v[b], c.window, c.n_sink, c.scale)
        # scores off by ds as in the attention (their size S; the lse adds |lse| <= S + log n to what
        # is rounded), weights by a relative 1.01 ds, sums of the rows and heads by 2^-23 each
        S = size.max() if size.size else 0.0
        ds = c.d * 2.0 ** -23 * S + (2 * S + np.log(n + 1) + 8) * 2.0 ** -22
        base = 0.75 * start[b, :n].double().cpu().numpy() if inout else 0.0
        tol = (1.01 * ds + (r * c.hkv * c.group + 32) * 2.0 ** -23) * w + 2.0 ** -22 * base + 2.0 ** -100
        assert (np.abs(got[b, :n] - (base + w)) <= tol).all(), b
        rest = start[b, n:].double().cpu().numpy() if inout else -7.0
        assert (got[b, n:] == rest).all()


# ------------------------------------------------------------------ eviction
def _scores(kind, B, n, g):
    s = torch.randn(B, n, generator=g)
    if kind == "ties":
        s = torch.randint(0, 3, (B, n), generator=g).float()
    elif kind == "same":
        s = torch.zeros(B, n)
        s[:, ::2] = -0.0
    elif kind == "odd":
        s = s.exp()
        s[:, ::5], s[:, 1::7], s[:, 2::11] = float("nan"), float("-inf"), float("inf")
    elif kind == "tiny":
        s = s * 1e-42
    return s


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", ["normal", "ties", "same", "odd", "tiny"])
@pytest.mark.parametrize("lens,budget,sink,recent,page", [
    ((50, 20, 7), 20, 2, 5, 16), ((300, 129, 1, 0), 128, 4, 32, 16), ((65, 64), 1, 0, 0, 16), ((65, 64), 1, 1, 0, 7),
    ((65, 64), 1, 0, 1, 1), ((2500, 1025, 3000), 1024, 4, 1020, 64), ((4000,), 2000, 0, 0, 33), ((40, 30), 50, 10, 10, 16),
    ((1500, 1300), 1299, 64, 100, 256)])
def test_eviction_keeps_what_the_oracle_keeps(lens, budget, sink, recent, page, kind, in_place):
    c = PagedCase(lens, (0,) * len(lens), page=page, hkv=2, d=64 if page == 7 else 128, spare=1).build()
    g = torch.Generator().manual_seed(budget + sink)
    B, n = len(lens), max(lens)
    host = _scores(kind, B, n + 2, g)
    score, most = host.cuda(), min(budget, n)
    kept = torch.full((B, budget), -9, dtype=torch.int32, device="cuda")
    new_len = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    before = [c.kd.cpu().clone(), c.vd.cpu().clone()]
    table, dst, out, k, v = c.table, None, score, c.kd, c.vd
    if not in_place:  # other pages of the same pool: the pool of a second set of pages behind it
        cols, total = -(-most // page), c.kd.shape[0]
        k, v = (torch.cat([x.contiguous(), torch.full((B * cols,) + x.shape[1:], float("nan"), dtype=x.dtype, device="cuda")])
                for x in (c.kd, c.vd))
        dst = (total + torch.randperm(B * cols, generator=g)).int().reshape(B, cols).cuda()
        out = torch.full((B, most + 1), -9.0, device="cuda")
        c.cache = type(c.cache)(k, v, n_q_heads=c.hkv * c.group)
        c.batch = c.cache.batch(c.table, c.lend, c.startd, c.n_rows, 0, c.max_len)
        table = dst
    c.cache.evict(c.batch, score, budget, kept, new_len, n_sink=sink, n_recent=recent, dst_table=dst, score_out=out)
    sync()
    for b in range(B):
        ids = P.evict(host[b].numpy(), lens[b], budget, sink, recent)
        m = len(ids)
        assert new_len[b].item() == m and kept[b, :m].tolist() == ids and (kept[b, m:] == -9).all()
        i = torch.arange(m)
        np.testing.assert_array_equal(out[b, :m].cpu().numpy(), host[b, ids].numpy())
        if not in_place:
            assert (out[b, m:] == -9).all()
        else:
            assert (out[b, m:lens[b]] == 0).all()
            np.testing.assert_array_equal(out[b, lens[b]:].cpu().numpy(), host[b, lens[b]:].numpy())
        for pool, was in zip((k, v), before):
            old = torch.tensor(ids, dtype=torch.long)
            want = was[c.table[b].cpu().long()[old // page], :, old % page]
            got = pool.cpu()[table[b].cpu().long()[i // page], :, i % page]
            assert torch.equal(got.contiguous().view(torch.int16), want.contiguous().view(torch.int16)), b
    if not in_place:
        total = before[0].shape[0]
        for pool, was in zip((k, v), before):   # the pages read are as they were
            assert torch.equal(pool[:total].cpu().view(torch.int16), was.contiguous().view(torch.int16))


def test_eviction_writes_the_new_lengths_over_the_old():
    c = PagedCase((90, 30, 200), (0, 0, 0)).build()
    score = torch.rand(3, 200, device="cuda")
    kept = torch.zeros(3, 50, dtype=torch.int32, device="cuda")
    c.cache.evict(c.batch, score, 50, kept, c.lend, n_recent=10)
    sync()
    assert c.lend.tolist() == [50, 30, 50]


# ------------------------------------------------------------------ together
def _step(c, k, v, out, lse, score, accepted):
    c.cache.append(c.batch, k, v)
    c.cache.attention(c.batch, c.qd, out, lse=lse)
    c.cache.weights(c.batch, c.qd, lse, score, score_in=score, rows_used=accepted)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("rows", [1, 5, 40])
def test_a_run_of_steps_with_evictions(rows, graph):
    """Several steps of append, attention and accumulation, then an eviction in place, against the
    oracle on a growing and shrinking list of slots; captured once and replayed in one variant."""
    c = PagedCase((rows + 50, rows + 131, rows), (rows, rows, rows), hkv=2, spare=40).build()
    B, width, t = 3, c.table.shape[1] * c.page, TYPES[c.dtype]
    total = B * c.table.shape[1]
    ids = torch.randperm(total, generator=torch.Generator().manual_seed(1)).int().reshape(B, -1).cuda()
    c.table.copy_(ids)
    k_pool = torch.full((total, c.hkv, c.page, c.d), float("nan"), dtype=t, device="cuda")
    v_pool = k_pool.clone()
    hist = []
    for b in range(B):
        n = c.lens[b] - rows
        kb, vb = (torch.from_numpy(x[b][:n]).to(t) for x in (c.k, c.v))
        j = torch.arange(n)
        for pool, x in ((k_pool, kb), (v_pool, vb)):
            pool[c.table[b].cpu().long()[j // c.page].cuda(), :, (j % c.page).cuda()] = x.cuda()
        hist.append([kb.double().numpy(), vb.double().numpy(), np.zeros(n)])
    c.cache = type(c.cache)(k_pool, v_pool, n_q_heads=c.hkv * c.group)
    c.batch = c.cache.batch(c.table, c.lend, c.startd, c.n_rows, rows, width)
    k = torch.empty(c.n_rows, c.hkv, c.d, dtype=t, device="cuda")
    v, q = torch.empty_like(k), c.qd
    out, lse = c.outputs()
    score = torch.zeros(B, width, device="cuda")
    accepted = torch.full((B,), rows, dtype=torch.int32, device="cuda")
    kept = torch.zeros(B, 90, dtype=torch.int32, device="cuda")
    lens = [c.lens[b] - rows for b in range(B)]
    g = torch.Generator().manual_seed(9)
    run = None
    for step in range(4):
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=g).to(t))
        for b in range(B):
            lens[b] += rows
        c.lend.copy_(torch.tensor(lens, dtype=torch.int32))
        if not graph:
            _step(c, k, v, out, lse, score, accepted)
        else:
            if run is None:
                run = torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(run):
                    _step(c, k, v, out, lse, score, accepted)
            run.replay()
        sync()
        c.lens, c.qf = tuple(lens), q.double().cpu().numpy()
        for b in range(B):
            s = slice(c.starts[b], c.starts[b] + rows)
            hist[b][0] = np.concatenate([hist[b][0], k[s].double().cpu().numpy()])
            hist[b][1] = np.concatenate([hist[b][1], v[s].double().cpu().numpy()])
            _, l, _, _ = P.attention(c.qf[s], hist[b][0], hist[b][1], 0, 0, c.scale)
            w = P.weights(c.qf[s], hist[b][0], l, rows, 0, 0, c.scale)
            hist[b][2] = np.concatenate([hist[b][2], np.zeros(rows)]) + w
            np.testing.assert_allclose(score[b, :lens[b]].cpu().numpy(), hist[b][2], rtol=1e-4, atol=1e-6)
        c.k, c.v = [h[0] for h in hist], [h[1] for h in hist]
        c.check_attention(out, lse)
        if step % 2:
            host = score.cpu().numpy()
            c.cache.evict(c.batch, score, 90, kept, c.lend, n_sink=2, n_recent=20, score_out=score)
            sync()
            for b in range(B):
                stay = P.evict(host[b], lens[b], 90, 2, 20)
                hist[b] = [h[stay] for h in hist[b]]
                lens[b] = len(stay)
                hist[b][2] = host[b][stay].astype(np.float64)
            assert c.lend.tolist() == lens


def test_two_streams_with_their_own_workspaces_and_two_graphs_sharing_one():
    c = PagedCase((700, 300), (1, 1), hkv=2).build()
    d = PagedCase((260, 500), (40, 60), hkv=2, seed=4).build()
    want = [x.attend() for x in (c, d)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [c.outputs(), d.outputs()]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, s, (o, l) in zip((c, d), streams, got):
            x.cache.attention(x.batch, x.qd, o, lse=l, stream=s)
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)
    big = max((c.batch, d.batch), key=lambda x: x.ws_bytes).workspace
    graphs = []
    for x in (c, d):
        x.batch = x.cache.batch(x.table, x.lend, x.startd, x.n_rows, x.max_rows, x.max_len, workspace=big)
        gr = torch.cuda.CUDAGraph()
        o, l = x.outputs()
        with torch.cuda.graph(gr):
            x.cache.attention(x.batch, x.qd, o, lse=l)
        graphs.append((gr, o, l))
    for _ in range(3):
        for gr, o, l in graphs:
            o.fill_(0)
            gr.replay()
        for (gr, o, l), (wo, wl) in zip(graphs, want):
            torch.cuda.synchronize()
            assert torch.equal(o, wo) and torch.equal(l, wl)
    sync()


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and more than 2^31 elements per pool side: the request's pages
    lie at its far end."""
    page, hkv, d = 64, 8, 128
    n_pages = (1 << 32) // (page * hkv * d) + 8          # just over 2^32 elements
    k = torch.empty(n_pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    c = PagedCase((200, 130), (1, 20), hkv=hkv, group=1, page=page).build()
    held = [-(-n // page) for n in c.lens]
    far = torch.arange(n_pages - 7, n_pages, device="cuda", dtype=torch.int32)
    table = torch.zeros_like(c.table)
    at = 0
    for b, h in enumerate(held):
        for i in range(h):
            k[far[at].item()] = c.kd[c.table[b, i].item()]
            v[far[at].item()] = c.vd[c.table[b, i].item()]
            table[b, i] = far[at]
            at += 1
    c.cache = type(c.cache)(k, v, n_q_heads=hkv)
    c.batch = c.cache.batch(table, c.lend, c.startd, c.n_rows, c.max_rows, c.max_len)
    out, lse = c.attend()
    sync()
    c.check_attention(out, lse)
    new = torch.randn(c.n_rows, hkv, d, device="cuda").to(torch.bfloat16)
    c.cache.append(c.batch, new, new)
    sync()
    assert torch.equal(k[table[1, 2].item(), :, 1], new[20])
    score, kept = torch.rand(2, 200, device="cuda"), torch.zeros(2, 100, dtype=torch.int32, device="cuda")
    c.cache.evict(c.batch, score, 100, kept, c.lend)
    sync()
    assert c.lend.tolist() == [100, 100]


def test_python_checks():
    from block_drafter_gb300.paged import PagedCache
    c = PagedCase((40, 50), (1, 2)).build()
    out, lse = c.outputs()
    for bad in (c.qd.float(), c.qd[:2], c.qd[:, :3], c.qd.transpose(1, 2)):
        with pytest.raises(ValueError):
            c.cache.attention(c.batch, bad, out)
    with pytest.raises(ValueError):
        c.cache.attention(c.batch, c.qd, out, lse=lse.double())
    with pytest.raises(ValueError):
        c.cache.attention(c.batch, c.qd.cpu(), out)
    with pytest.raises(RuntimeError, match="overlap"):
        c.cache.attention(c.batch, c.qd, c.qd)
    with pytest.raises(ValueError):
        c.cache.batch(c.table.long(), c.lend, c.startd, 3, 2, 50)
    with pytest.raises(ValueError):
        c.cache.batch(c.table, c.lend, None, 3, 2, 50)
    with pytest.raises(RuntimeError, match="max_len"):
        t = c.cache.batch(c.table, c.lend, c.startd, 3, 2, 10 ** 6)
        c.cache.attention(t, c.qd, out)
    with pytest.raises(ValueError):
        c.cache.evict(c.batch, lse, 10, c.table, c.lend)
    with pytest.raises(RuntimeError, match="workspace"):
        t = c.cache.batch(c.table, c.lend, c.startd, 3, 2, 50, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
        c.cache.attention(t, c.qd, out)
    assert isinstance(c.cache, PagedCache)


@pytest.mark.parametrize("rows,group,hkv,window,n_sink,d,dtype", [
    (16, 4, 8, 0, 0, 128, "bf16"), (64, 4, 2, 0, 0, 128, "fp16"), (100, 1, 3, 0, 0, 64, "bf16"), (65, 2, 1, 40, 3, 64, "fp16"),
    (33, 8, 9, 100, 130, 128, "bf16"), (129, 16, 1, 1, 0, 128, "bf16"), (70, 3, 2, 50, 4, 128, "bf16"), (8, 128, 2, 0, 0, 64, "fp16"),
    (300, 4, 1, 129, 1, 64, "bf16")])
@pytest.mark.parametrize("page", [8, 33, 64])
def test_weights_of_many_rows(rows, group, hkv, window, n_sink, d, dtype, page):
    """The row counts from which the tensor-core form takes over, and the forms that it leaves."""
    c = PagedCase((rows + 260, 257, max(1, rows - 5)), (rows, min(rows, 40), rows), hkv=hkv, group=group, d=d, dtype=dtype, page=page,
                  window=window, n_sink=n_sink, lead=1, seed=rows).build()
    _, lse = c.attend()
    used = (rows, 0, max(1, rows - 7))
    score = torch.full((3, c.max_len), -7.0, device="cuda")
    c.cache.weights(c.batch, c.qd, lse, score, rows_used=torch.tensor(used, dtype=torch.int32, device="cuda"), window=window, n_sink=n_sink)
    sync()
    got, lse = score.double().cpu().numpy(), lse.double().cpu().numpy()
    for b, (n, r) in enumerate(zip(c.lens, c.rows)):
        s = slice(c.starts[b], c.starts[b] + r)
        w = P.weights(c.qf[s], c.k[b], lse[s], used[b], window, n_sink, c.scale)
        _, _, _, size = P.attention(c.qf[s], c.k[b], c.v[b], window, n_sink, c.scale)
        S = size.max()      # the tolerance of test_weights_match_the_oracle
        ds = c.d * 2.0 ** -23 * S + (2 * S + np.log(n + 1) + 8) * 2.0 ** -22
        tol = (1.01 * ds + (r * hkv * group + 32) * 2.0 ** -23) * w + 2.0 ** -100
        assert (np.abs(got[b, :n] - w) <= tol).all(), b
        assert (got[b, n:] == -7.0).all()


@pytest.mark.parametrize("rows", [2, 40])
def test_weights_of_hidden_garbage(rows):
    """NaN keys in a slot, NaN in a row that does not count: other slots and rows stand."""
    case = PagedCase((300,), (rows,), hkv=2).build()
    _, lse = case.attend()
    clean, score = (torch.zeros(1, 300, device="cuda") for _ in range(2))
    used = torch.tensor([rows - 1], dtype=torch.int32, device="cuda")
    case.cache.weights(case.batch, case.qd, lse, clean, rows_used=used)
    case.kd[case.table[0, 3].item(), :, 5] = float("nan")     # slot 53, seen by every row
    case.qd[rows - 1] = float("nan")
    lse[rows - 1] = float("nan")
    case.cache.weights(case.batch, case.qd, lse, score, rows_used=used)
    sync()
    assert torch.isnan(score[0, 53])
    keep = torch.arange(300, device="cuda") != 53
    assert torch.equal(score[0, keep], clean[0, keep])


def test_a_long_list_of_items_is_planned_apart():
    """More requests and row tiles than a block of the tensor-core attention sums up by itself."""
    rows = [1] * 130
    rows[7], rows[60], rows[129] = 600, 90, 300
    lens = [r + (i * 37) % 190 for i, r in enumerate(rows)]
    c = PagedCase(tuple(lens), tuple(rows), hkv=1, group=8, d=64).build()
    out, lse = c.attend()
    sync()
    c.check_attention(out, lse)


@pytest.mark.parametrize("rows", [1, 7, 300])
def test_rows_that_see_garbage_show_it_and_others_do_not(rows):
    """NaN among the visible values of every row (no hidden garbage): the affected column alone."""
    c = PagedCase((700,), (rows,), hkv=2, group=2).build()
    c.vd[c.table[0, 2].item(), 1, 9, 5] = float("nan")        # slot 41, KV head 1
    out, lse = c.attend()
    sync()
    bad = torch.zeros(c.n_rows, 4, c.d, dtype=torch.bool, device="cuda")
    bad[:, 2:, 5] = True
    assert torch.equal(torch.isnan(out), bad) and torch.isfinite(lse).all()


def test_weights_on_two_streams_beside_attention():
    """Calls that share the SMs: clusters that wait for TMEM must not wait for each other."""
    cases = [PagedCase((900, 700), (200, 150), hkv=8, group=4, d=64, page=64, seed=s).build() for s in (1, 2)]
    lse = [c.attend()[1] for c in cases]
    want = [torch.zeros(2, c.max_len, device="cuda") for c in cases]
    got = [torch.zeros_like(w) for w in want]
    for c, l, w in zip(cases, lse, want):
        for _ in range(20):
            c.cache.weights(c.batch, c.qd, l, w, score_in=w)
    out, l3 = cases[0].outputs()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, l, x, s in zip(cases, lse, got, streams):
            c.cache.weights(c.batch, c.qd, l, x, score_in=x, stream=s)
        cases[0].cache.attention(cases[0].batch, cases[0].qd, out, lse=l3, stream=streams[2])
    sync()
    for x, w in zip(got, want):
        assert torch.equal(x, w)
    assert torch.equal(l3, lse[0])


def test_a_workspace_must_be_contiguous():
    c = PagedCase((40,), (1,)).build()
    n = c.batch.ws_bytes
    for bad in (torch.empty(1, dtype=torch.uint8, device="cuda").expand(n), torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            c.cache.batch(c.table, c.lend, c.startd, c.n_rows, c.max_rows, c.max_len, workspace=bad)


@pytest.mark.parametrize("lens,rows,kw,slack", [
    ((1500,), (1500,), dict(), 0),                                  # two rounds of items
    ((1400,), (1200,), dict(lead=300), 500),                        # bounds beyond the lengths
    ((900, 700, 1100, 640), (640,) * 4, dict(d=64, dtype="fp16"), 0),   # equal rows, other lengths
    ((1000, 0, 300), (500,) * 3, dict(group=8), 0),                 # no slots; rows before the first slot
    ((1300,), (1300,), dict(window=200, n_sink=5, page=24), 0),
    ((1100, 1100), (1, 1100), dict(), 0),                           # not equal: shared out
])
def test_prompts_whose_items_are_not_shared(lens, rows, kw, slack):
    c = PagedCase(lens, rows, **{**dict(hkv=8, group=4), **kw}).build()
    if slack:
        c.batch = c.cache.batch(c.table, c.lend, c.startd, c.n_rows, c.max_rows + slack, c.max_len)
    out, lse = c.attend()
    sync()
    c.check_attention(out, lse)
    c.check_guards(out, lse)


@pytest.mark.parametrize("n,rows,group,d,dtype", [(40, 1, 1, 64, "bf16"), (44, 2, 2, 128, "fp16"), (21, 5, 3, 64, "fp16")])
def test_few_rows_of_many_heads_share_the_blocks(n, rows, group, d, dtype):
    lens = tuple((i * 389) % 900 + (i % 3) for i in range(n))
    c = PagedCase(lens, tuple((i % rows) + 1 for i in range(n)), hkv=8, group=group, d=d, dtype=dtype).build()
    out, lse = c.attend()
    sync()
    c.check_attention(out, lse)
    c.check_guards(out, lse)


@pytest.mark.parametrize("lens,rows,kw", [
    ((4100,), (1,), dict(hkv=8)),                                        # sixteen blocks a head
    ((2300, 3, 0, 17), (2, 4, 1, 4), dict(hkv=4)),                       # fewer units than blocks, no slot
    ((1900, 1200), (5, 4), dict(hkv=5, group=3, d=64, dtype="fp16")),    # up to 15 rows, eight blocks a head
    ((9000, 700, 5000), (1, 1, 1), dict(hkv=8, window=1500, n_sink=3, page=24)),
])
def test_few_rows_of_few_heads_are_a_clusters(lens, rows, kw):
    c = PagedCase(lens, rows, **kw).build()
    out, lse = c.attend()
    sync()
    c.check_attention(out, lse)
    again, lse2 = c.attend()
    sync()
    assert torch.equal(again[c.starts[0]:c.starts[-1]], out[c.starts[0]:c.starts[-1]]) and torch.equal(lse2, lse)


def test_hidden_garbage_of_a_clusters_head():
    c = PagedCase((3000, 2000), (4, 4), hkv=2, group=2, window=700).build()
    want, wl = c.attend()
    for b, n in enumerate(c.lens):      # slots that the later rows see no more, and those that the first do not yet
        for j in list(range(n - 704, n - 700)) + list(range(n - 3, n)):
            c.vd[c.table[b, j // c.page].item(), :, j % c.page] = float("inf")
    out, lse = c.attend()
    sync()
    assert torch.equal(lse, wl)
    bad = torch.isfinite(out).logical_not().flatten(1).any(1)
    assert bad.tolist() == [True] * 8   # each row sees one of them or more


@pytest.mark.parametrize("lens,rows,kw", [
    ((4100,), (16,), dict(hkv=8)),                                           # eight blocks an item, shared streams
    ((2600,), (33,), dict(hkv=4, group=5, page=33)),                         # 165 rows: items of 128
    ((2000, 30, 0, 5), (20, 9, 3, 9), dict(hkv=3, group=7, d=64, dtype="fp16")),   # no tile for most blocks, no slot
    ((3000,), (300,), dict(hkv=2, group=1, dtype="fp16")),
    ((5000, 900), (40, 200), dict(hkv=2, group=2, window=1100, n_sink=4, page=24)),
    ((129, 257), (128, 128), dict(hkv=1, group=2, d=64)),
    ((6000,), (256,), dict(hkv=1, group=1, page=64)),                        # two streams, sixteen blocks
])
def test_items_of_a_cluster(lens, rows, kw):
    c = PagedCase(lens, rows, lead=2, **kw).build()
    out, lse = c.attend()
    sync()
    c.check_attention(out, lse)
    c.check_guards(out, lse)
    again, lse2 = c.attend()
    sync()
    s = slice(c.starts[0], c.starts[-1])
    assert torch.equal(again[s], out[s]) and torch.equal(lse2, lse)


def test_hidden_garbage_of_a_clusters_item():
    """Infinities among the last slots, which all rows but the request's last do not see."""
    c = PagedCase((3001,), (30,), hkv=2, group=4).build()
    want, wl = c.attend()
    c.vd[c.table[0, 3000 // c.page].item(), :, 3000 % c.page] = float("inf")
    out, lse = c.attend()
    sync()
    assert torch.equal(lse, wl) and not torch.isfinite(out[29]).any()
    c.check_attention(torch.where(torch.isfinite(out), out, want), lse)
    assert torch.isfinite(out[:29]).all()


@pytest.mark.parametrize("rows,group,hkv,window,n_sink,d,dtype", [
    (3, 5, 8, 0, 0, 128, "bf16"), (1, 11, 3, 90, 2, 64, "fp16"), (12, 5, 2, 0, 0, 64, "bf16"), (1, 48, 2, 0, 0, 128, "fp16"),
    (9, 7, 9, 60, 3, 128, "fp16"), (200, 7, 1, 0, 0, 128, "bf16"), (2, 100, 1, 0, 0, 64, "bf16")])
def test_weights_of_groups_that_do_not_fill_a_row_tile(rows, group, hkv, window, n_sink, d, dtype):
    test_weights_of_many_rows(rows, group, hkv, window, n_sink, d, dtype, 16)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens,budget,sink,recent,page,kind", [
    ((20000, 9000, 300), 8191, 4, 512, 16, "normal"), ((8193,), 100, 0, 0, 64, "ties"), ((16383, 12345), 12345, 3, 0, 33, "odd"),
    ((70001, 66000), 5000, 1, 4000, 256, "same"), ((70001,), 65999, 0, 17, 64, "normal")])
def test_eviction_of_long_requests(lens, budget, sink, recent, page, kind, in_place):
    """Selections by eight blocks, and of more slots than their registers hold."""
    test_eviction_keeps_what_the_oracle_keeps(lens, budget, sink, recent, page, kind, in_place)


@pytest.mark.parametrize("rows", [1, 40])
def test_a_short_request_under_a_large_bound(rows):
    """A batch made for long contexts, as a captured step has it, with few slots yet."""
    c = PagedCase((70,), (rows,), hkv=8, page=64).build()
    table = torch.zeros(1, 512, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    for max_len in (600, 5000, 32768):
        c.batch = c.cache.batch(table, c.lend, c.startd, c.n_rows, c.max_rows, max_len)
        out, lse = c.attend()
        sync()
        c.check_attention(out, lse)


def _give_back_unseen_pages(c):
    """Page-table entries of pages no slot of which a row sees: as a program leaves them behind a window."""
    given = 0
    for b, (n, r) in enumerate(zip(c.lens, c.rows)):
        seen = P.visible(n, r, c.window, c.n_sink).any(0)
        for i in range(-(-n // c.page)):
            if not seen[i * c.page:(i + 1) * c.page].any():
                c.table[b, i] = (-1, 2 ** 30, c.kd.shape[0])[i % 3]
                given += 1
    assert given > 0


@pytest.mark.parametrize("page", [8, 16, 33, 64])
@pytest.mark.parametrize("rows,kw", [
    (1, dict()), (4, dict(hkv=1)), (16, dict()), (40, dict(d=64, dtype="fp16")), (150, dict(group=2)), (9, dict(group=40, hkv=1))])
def test_pages_that_no_row_sees_may_be_given_back(rows, kw, page):
    c = PagedCase((1000, 701), (rows, max(1, rows - 1)), page=page, window=200, n_sink=3, **kw).build()
    want, wl = c.attend()
    ws = torch.zeros(2, c.max_len, device="cuda")
    c.cache.weights(c.batch, c.qd, wl, ws, window=c.window, n_sink=c.n_sink)
    sync()
    _give_back_unseen_pages(c)
    out, lse = c.attend()
    sync()                                  # nothing is reported
    assert torch.equal(out, want) and torch.equal(lse, wl)
    score = torch.zeros_like(ws)
    c.cache.weights(c.batch, c.qd, lse, score, window=c.window, n_sink=c.n_sink)
    sync()
    assert torch.equal(score, ws)
    # rows done again for an infinity among the values they do not see look past such pages, too
    c.vd[c.table[0, 999 // page].item(), :, 999 % page] = float("inf")
    out, _ = c.attend()
    sync()
    assert torch.isfinite(out[:rows - 1]).all() and not torch.isfinite(out[rows - 1]).any()


@pytest.mark.parametrize("rows", [1, 16, 150])
@pytest.mark.parametrize("page", [16, 33])
def test_a_seen_page_outside_the_pool_is_still_reported(rows, page):
    from block_drafter_gb300 import binding as B
    c = PagedCase((1000,), (rows,), page=page, window=200, n_sink=3).build()
    _, lse = c.attend()
    score = torch.zeros(1, c.max_len, device="cuda")
    sync()
    for slot in (0, 1000 - rows - 199, 999):            # a sink, the first row's window's first slot, the last slot
        keep = c.table[0, slot // page].item()
        c.table[0, slot // page] = -1
        for call in (lambda: c.attend(), lambda: c.cache.weights(c.batch, c.qd, lse, score, window=200, n_sink=3)):
            call()
            with pytest.raises(B.BdError):
                B.sync_status()
        c.table[0, slot // page] = keep
    c.attend()
    sync()


@pytest.mark.parametrize("lens,rows,kw,bound", [
    ((300,), (1,), dict(), 0),                                       # a head is one block's: its four warps
    ((4100,), (1,), dict(hkv=8), 0),                                 # a cluster's
    ((3000, 5000, 4000), (1, 1, 1), dict(hkv=8), 40000),             # shared out, joined by a launch
    ((3000, 5000, 4000), (4, 3, 4), dict(hkv=8, dtype="fp16"), 40000),
    ((700,), (16,), dict(), 0),                                      # a block of rows: the two streams
    ((4100,), (16,), dict(hkv=8), 0),                                # a cluster's item
    ((4100,), (150,), dict(group=2, d=64, dtype="fp16"), 0),
    ((3000, 5000, 4000), (16, 9, 16), dict(hkv=8), 40000),           # items shared out
])
def test_a_visible_nan_beside_a_slot_that_outweighs_it_shows(lens, rows, kw, bound):
    """One key outweighs every other by more than any exponent holds; NaN values far from it, each in a column of
    its own, still make that column NaN, whichever warp, stream or block has them."""
    c = PagedCase(lens, rows, spare=-(-bound // 16), **kw).build()
    if bound:
        c.batch = c.cache.batch(c.table, c.lend, c.startd, c.n_rows, c.max_rows, bound)
    c.qd.fill_(1.0)
    bad = np.zeros((c.n_rows, c.hkv * c.group, c.d), bool)
    for b, (n, r) in enumerate(zip(lens, rows)):
        at = lambda j: (c.table[b, j // c.page].item(), slice(None), j % c.page)
        c.kd[at(n // 2)] = 32.0                # scale q.k = 32 sqrt(D): 256 and more beyond the others' few
        see = P.visible(n, r, 0, 0)
        for col, j in enumerate(range(n - 1, -1, -(n // 48 + 1))):
            if j != n // 2:
                c.vd[at(j)][:, col] = float("nan")
                bad[c.starts[b]:c.starts[b] + r, :, col] = see[:, j, None]
    out, lse = c.attend()
    sync()
    assert bad.any() and np.array_equal(torch.isnan(out).cpu().numpy(), bad) and torch.isfinite(lse).all()


@pytest.mark.parametrize("rows,window,kw,launches", [
    (4, 700, dict(group=2, hkv=2), 1),              # few rows: a head is a cluster's
    (4, 700, dict(group=2, hkv=64), 2),             # shared out, joined by a launch
    (16, 700, dict(group=4, hkv=2), 1),             # an item is a cluster's
    (17, 2600, dict(group=1, hkv=51), 2),           # items shared out
])
@pytest.mark.parametrize("hit", ["last", "first"])
def test_rows_done_again_hold_what_they_see_alone(rows, window, kw, launches, hit):
    """Infinities in a slot that one row alone sees, the last row's own or the first one of the first row's window: that row
    shows them, and every other one, done again, agrees with the oracle and keeps its lse."""
    from block_drafter_gb300 import binding as B
    c = PagedCase((3000, 2900, 3100), (rows,) * 3, window=window, **kw).build()
    before = B.kernel_launches()
    want, wl = c.attend()
    assert B.kernel_launches() - before == launches
    mine = []
    for b, n in enumerate(c.lens):
        j = n - 1 if hit == "last" else n - rows - window + 1
        c.vd[c.table[b, j // c.page].item(), :, j % c.page] = float("inf")
        mine.append(c.starts[b] + (rows - 1 if hit == "last" else 0))
    out, lse = c.attend()
    sync()
    assert torch.equal(lse, wl)
    fine = torch.isfinite(out).flatten(1)
    assert [i for i in range(c.n_rows) if not fine[i].any()] == mine and fine.all(1).sum().item() == c.n_rows - 3
    c.check_attention(torch.where(torch.isfinite(out), out, want), lse)


def test_a_batchs_workspace_waits_for_the_streams_it_is_used_on():
    c = PagedCase((700, 300), (40, 60)).build()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for how in ("given", "current"):
        c.batch = c.cache.batch(c.table, c.lend, c.startd, c.n_rows, c.max_rows, c.max_len)
        out, lse = c.outputs()
        torch.cuda.synchronize()
        s, n, place = torch.cuda.Stream(), c.batch.ws_bytes, c.batch.ws_ptr
        with torch.cuda.stream(s):
            torch.cuda._sleep(200_000_000)      # about 0.1 s
            if how == "current":
                c.cache.attention(c.batch, c.qd, out, lse=lse)
        if how == "given":
            c.cache.attention(c.batch, c.qd, out, lse=lse, stream=s)
        c.batch = None                          # its call has not begun
        other = torch.empty(n, dtype=torch.uint8, device="cuda")
        assert other.data_ptr() != place
        other.fill_(255)
        sync()
        torch.cuda.synchronize()
        c.check_attention(out, lse)
        del other
        torch.cuda.empty_cache()


def test_a_batchs_workspace_waits_for_the_stream_it_was_allocated_on():
    import time
    c = PagedCase((700, 300), (40, 60)).build()
    out, lse = c.outputs()
    s, home, done = torch.cuda.Stream(), torch.cuda.Event(), torch.cuda.Event()
    torch.cuda.synchronize()
    torch.cuda._sleep(1_000_000_000)            # about 0.5 s: what the memory was before may still be in use
    home.record()
    c.batch = c.cache.batch(c.table, c.lend, c.startd, c.n_rows, c.max_rows, c.max_len)
    c.cache.attention(c.batch, c.qd, out, lse=lse, stream=s)
    done.record(s)
    time.sleep(0.05)
    early = done.query()
    assert home.query() or not early
    torch.cuda.synchronize()
    sync()
    c.check_attention(out, lse)
    # a batch made before, captured and replayed on streams of its own
    graph = torch.cuda.CUDAGraph()
    c.batch = c.cache.batch(c.table, c.lend, c.startd, c.n_rows, c.max_rows, c.max_len)
    o2, l2 = c.outputs()
    with torch.cuda.graph(graph):
        c.cache.attention(c.batch, c.qd, o2, lse=l2)
    with torch.cuda.stream(s):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("requests,hkv,bound,window,launches", [
    (1, 1, 16384, 0, 1), (1, 1, 32768, 0, 2), (1, 2, 16384, 0, 1), (1, 2, 32768, 0, 2), (1, 4, 16384, 0, 1), (1, 4, 32768, 0, 2),
    (1, 8, 16384, 0, 1), (1, 8, 32768, 0, 2), (1, 16, 4096, 0, 1), (1, 16, 16384, 0, 2),
    (5, 8, 32768, 8192, 1), (10, 8, 32768, 4096, 1), (19, 8, 32768, 4096, 1), (2, 1, 32768, 32000, 2), (8, 1, 16384, 0, 1), (2, 8, 16384, 0, 2)])
def test_a_token_is_shared_out_where_that_was_faster(requests, hkv, bound, window, launches):
    """A cluster a head is one launch, equal shares and their joins are two; which was measured to be faster at the bound."""
    from block_drafter_gb300 import binding as B
    c = PagedCase(tuple(40 + 30 * b for b in range(requests)), (1,) * requests, hkv=hkv, window=window, spare=-(-bound // 16)).build()
    c.batch = c.cache.batch(c.table, c.lend, c.startd, c.n_rows, 1, bound)
    before = B.kernel_launches()
    out, lse = c.attend()
    assert B.kernel_launches() - before == launches
    sync()
    c.check_attention(out, lse)


@pytest.mark.parametrize("lens,rows,kw", [
    ((32768,), (1,), dict(hkv=1)), ((20011,), (1,), dict(hkv=1, group=16, d=64)), ((12001, 30000), (2, 1), dict(hkv=1, dtype="fp16")),
    ((32768,), (1,), dict(hkv=2, page=64)), ((17000,), (4,), dict(hkv=2, d=64, page=33)), ((19999,), (60,), dict(hkv=1)),
    ((23000,), (16,), dict(hkv=2, dtype="fp16", page=64))])
def test_few_heads_over_long_requests(lens, rows, kw):
    c = PagedCase(lens, rows, **kw).build()
    out, lse = c.attend()
    sync()
    c.check_attention(out, lse)


@pytest.mark.parametrize("in_place", [True, False])
def test_keys_and_values_in_one_pool(in_place):
    """One pool for both: a row is its key and its value; long in-place moves keep their slots."""
    lens, budget, page = (20000, 9000), 8000, 16
    c = PagedCase(lens, (3, 70), page=page, hkv=4, d=64).build()
    x = c.kd.clone() if in_place else torch.cat([c.kd, torch.full((1000,) + c.kd.shape[1:], float("nan"), dtype=c.kd.dtype, device="cuda")])
    c.cache = type(c.cache)(x, x, n_q_heads=c.hkv * c.group)
    c.batch = c.cache.batch(c.table, c.lend, c.startd, c.n_rows, c.max_rows, c.max_len)
    new = torch.randn(c.n_rows, c.hkv, c.d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    rows = new.cuda()
    c.cache.append(c.batch, rows, rows)
    for b, (n, r) in enumerate(zip(c.lens, c.rows)):
        c.k[b][n - r:] = new[c.starts[b]:c.starts[b] + r].double().numpy()
    c.v = c.k
    out, lse = c.attend()
    sync()
    c.check_attention(out, lse)
    score = torch.rand(2, max(lens), device="cuda")
    kept = torch.zeros(2, budget, dtype=torch.int32, device="cuda")
    new_len = torch.zeros(2, dtype=torch.int32, device="cuda")
    dst = None if in_place else (c.kd.shape[0] + torch.arange(1000, device="cuda", dtype=torch.int32)).view(2, 500)
    c.cache.evict(c.batch, score, budget, kept, new_len, dst_table=dst)
    sync()
    table = c.table if in_place else dst
    for b in range(2):
        i = torch.arange(budget, device="cuda")
        got = x[table[b].long()[i // page], :, i % page]
        assert new_len[b].item() == budget and torch.equal(got.double().cpu(), torch.from_numpy(c.k[b])[kept[b].cpu().long()])


@pytest.mark.parametrize("n,group", [(40, 1), (40, 8), (40, 12), (200, 4), (200, 16)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_few_rows_keep_the_rest_of_their_weights(n, group, dtype):
    """Values that cancel: the weights' rounding to 16 bits, about as large as the output's own where they do not,
    would stand out.  Tolerance: that of check_attention with the weights as a 16-bit part and a 16-bit rest (u^2 for u;
    what fp16 loses below its subnormals, 2^-25 of weights formed 2^12 above the largest's size, is 2^-37 a slot)."""
    c = PagedCase((n,), (1,), hkv=2, group=group, dtype=dtype).build()
    t = TYPES[dtype]
    u = torch.finfo(t).eps / 2
    q = (torch.randn(1, 2, 1, c.d, generator=torch.Generator().manual_seed(n + group)) * 0.05).to(t).expand(1, 2, group, c.d)
    c.qd.copy_(q.reshape(1, -1, c.d).cuda())
    qf, lost = q.double().numpy(), np.zeros((1, 2 * group, c.d))
    for h in range(2):                                  # the last slot's value cancels the others' sum
        s = c.scale * (c.k[0][:, h] @ qf[0, h, 0])
        w = np.exp(s - s.max())
        last = -(w[:-1, None] * c.v[0][:-1, h]).sum(0) / w[-1]
        c.v[0][-1, h] = torch.from_numpy(last).to(t).double().numpy()
        c.vd[c.table[0, (n - 1) // c.page].item(), h, (n - 1) % c.page] = torch.from_numpy(last).to(t).cuda()
        lost[0, h * group:(h + 1) * group] = (torch.from_numpy(w).to(t).double().numpy() @ c.v[0][:, h]) / w.sum()
    ref, _, spread, size = P.attention(qf.reshape(1, -1, c.d), c.k[0], c.v[0], 0, 0, c.scale)
    ds = ((c.d * 2.0 ** -23) * size + (size + 4) * 2.0 ** -22)[..., None]
    tol = u * np.abs(ref) + torch.finfo(t).smallest_normal * u + (u * u + 2.02 * ds + (n + 64) * 2.0 ** -23) * spread + \
        n * 2.0 ** -37 * np.abs(c.v[0]).max()
    assert (np.abs(lost - ref) > tol).any()             # weights of 16 bits alone would fail here
    out, _ = c.attend()
    sync()
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
