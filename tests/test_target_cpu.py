"""The target-side operators without a GPU: the oracle's closed cases and the calls the library refuses."""
import numpy as np
import pytest
import torch

from oracle import target_oracle as T


@pytest.fixture(scope="module")
def B():
    from block_drafter_gb300 import builder
    builder.build()
    from block_drafter_gb300 import binding
    binding.lib()
    return binding


# ------------------------------------------------------------------ oracle
def test_4_bit_codes_by_hand():
    x = np.zeros(16)
    x[:10] = [6, -6, 0.25, 0.75, -1.25, 1.75, 2.5, 3.5, 5.0, 0.26]
    codes, scales = T.encode4(x)
    assert scales.tolist() == [0x38]                                    # 1.0
    code = np.stack((codes & 15, codes >> 4), -1).reshape(-1)
    assert code[:10].tolist() == [7, 15, 0, 2, 8 + 2, 4, 4, 6, 6, 1]
    assert T.decode4(codes, scales)[:10].tolist() == [6, -6, 0, 1, -1, 2, 2, 4, 4, 0.5]
    assert T.encode4(x * 8, 3)[0].tolist() == codes.tolist() and T.decode4(codes, scales, 3)[1] == -48
    assert T.encode4(np.full(16, 1e9))[1].tolist() == [126]             # 448, saturated
    assert T.encode4(np.full(16, np.nan))[1].tolist() == [0]
    assert T.encode4(np.full(16, -2.0 ** -20))[0].tolist() == [0] * 8   # below the smallest scale


def test_4_bit_numbers_are_torchs():
    every = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert (every == T.E4M3).all()
    x = torch.rand(4000, generator=torch.Generator().manual_seed(0)) * 500
    assert (T.nearest(T.E4M3, x.double().numpy()) == x.clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()).all()


def test_plan_by_hand():
    table = np.array([[9, 8, 7, -1], [5, -1, -1, -1], [4, 3, -1, -1]], dtype=np.int32)
    p = T.plan([4, 4, 1], [1, 5, 1], [3, 1, 2], table, [1, 2], 4, 8, True)
    assert p["seq_len"] == [5, 9, 2] and p["row_start"] == [0, 1, 6, 7] and p["held"] == [2, 3, 1]
    assert p["table"][1].tolist() == [5, 3, 7, -1] and p["free"] == [1, 2] and p["short"] == 0
    assert p["slot"].tolist() == [32, 12, 13, 14, 15, 28, 17, -1] and p["request"].tolist() == [0, 1, 1, 1, 1, 1, 2, -1]
    p = T.plan([4, 4, 1], [1, 9, 5], [3, 1, 2], table, [], 4, 15, False)
    assert p["short"] == 1 and p["seq_len"] == [5, 0, 6] and p["held"] == [3, 1, 2]


def test_rotation_by_hand():
    x = np.ones((1, 1, 4))
    y = T.head_norm_rope(x, None, 0.0, [np.pi / 2, 0.0], [1], False)
    np.testing.assert_allclose(y[0, 0], [-1, 1, 1, 1], atol=1e-15)
    y = T.head_norm_rope(x, [1, 2, 3, 4], 0.0, [np.pi / 2], [1], True)
    np.testing.assert_allclose(y[0, 0], [-2, 1, 3, 4], atol=1e-15)


def test_logprobs_by_hand():
    lp, ent, lse, ids, top = T.token_logprobs([0.0, 0.0, -np.inf, 0.0], [0, 2, -1], 1.0, 3)
    np.testing.assert_allclose([lp[0], ent, lse], [-np.log(3), np.log(3), np.log(3)])
    assert lp[1] == -np.inf and lp[2] == 0 and ids == [0, 1, 3]
    np.testing.assert_allclose(T.token_logprobs([1.0, 3.0], [1], 2.0, 0)[0], [-np.log1p(np.exp(-1))])


# ------------------------------------------------------------------ refusals
def _plan(B, **kw):
    pages = dict(n_requests=2, table_width=4, page_size=16, n_free=20, page_table=0x10000, held=0x11000, held_out=0x11000, free_pages=0x12000,
                 free_count=0x13000, free_count_out=0x13000)
    args = dict(len=0x20000, n_new=0x21000, n_rows=8, seq_len=0x22000, row_start=0x23000, row_request=0x24000, row_pos=0x25000, slot_map=0x26000,
                n_short=0x27000)
    for k, v in kw.items():
        (pages if k in pages else args)[k] = v
    a = args
    return B.lib().bd_paged_plan(B.PagedPages(**pages), a["len"], a["n_new"], 1, a["n_rows"], a["seq_len"], a["row_start"], a["row_request"],
                                 a["row_pos"], a["slot_map"], a["n_short"], None)


@pytest.mark.parametrize("kw,msg", [
    (dict(n_requests=0), b"n_requests"), (dict(n_requests=1025), b"n_requests"), (dict(table_width=0), b"table_width"),
    (dict(page_size=0), b"page_size"), (dict(n_free=0), b"n_free"), (dict(n_rows=-1), b"n_rows"), (dict(n_rows=2 ** 29), b"n_rows"),
    (dict(len=None), b"len must"), (dict(n_new=0x21002), b"n_new must"), (dict(held=None), b"held must"), (dict(page_table=None), b"page_table must"),
    (dict(free_pages=0x12001), b"free_pages must"), (dict(free_count_out=None), b"free_count_out must"), (dict(seq_len=None), b"seq_len must"),
    (dict(row_pos=None), b"row_pos must"), (dict(slot_map=0x26004), b"slot_map must"), (dict(seq_len=0x20004), b"overlap"),
    (dict(held_out=0x11004), b"overlap"), (dict(row_start=0x22004), b"overlap"), (dict(slot_map=0x25000), b"overlap"),
    (dict(n_short=0x13000), b"overlap"), (dict(held_out=0x10010), b"overlap"), (dict(page_table=0x12000 - 28), b"overlap"),
    (dict(row_request=0x25010), b"overlap"), (dict(free_count=0x1200c), b"overlap")])
def test_bad_plans_are_refused(B, kw, msg):
    assert _plan(B, **kw) == -1 and msg in B.lib().bd_last_error()


def test_a_null_plan_is_refused(B):
    assert B.lib().bd_paged_plan(None, *[None] * 2, 1, 0, *[None] * 7) == -1


def _kv4(B, **kw):
    c = B.Paged4Kv(8, 2, 128, B.BF16, 16, 10, 0, 0, 2 * 16 * 64, 16 * 64, 64, 2 * 16 * 8, 16 * 8, 8, 0x10000, 0x20000, 0x30000, 0x38000)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _batch(B, **kw):
    t = B.PagedBatch(2, 8, 4, 2, 100, 0x50000, 0x51000, 0x52000)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _attend4(B, kv, bt, q=0x60000, qs=1024, out=0x80000, os=1024, lse=None, window=0, sink=0, scale=0.1, ws=0x100000, n=1 << 40):
    return B.lib().bd_paged4_attention(kv, bt, q, qs, out, os, lse, window, sink, scale, ws, n, None)


def _append4(B, kv, bt, k=0x60000, ks=256, v=0x70000, vs=256, kh=None, vh=None):
    return B.lib().bd_paged4_append(kv, bt, k, ks, v, vs, kh, vh, None)


@pytest.mark.parametrize("field,val,status,msg", [
    ("dtype", 1, -2, b"dtype"), ("head_dim", 96, -2, b"head_dim"), ("head_dim", 256, -2, b"head_dim"), ("n_q_heads", 7, -1, b"multiple"),
    ("n_q_heads", 258, -2, b"128 query heads"), ("page_size", 0, -1, b"page_size"), ("n_pages", 0, -1, b"n_pages"), ("k", None, -1, b"pools"),
    ("v", 0x20008, -1, b"aligned"), ("k_scale", None, -1, b"k_scale"), ("v_scale", 0x38004, -1, b"aligned"), ("slot_stride", 72, -1, b"multiples of 16"),
    ("page_stride", -16, -1, b">= 0"), ("head_stride", 48, -1, b"at least"), ("slot_stride", 0, -1, b"at least"), ("scale_slot_stride", 12, -1, b"multiples"),
    ("scale_head_stride", 0, -1, b"at least"), ("scale_page_stride", -8, -1, b">= 0"), ("k_exp", 65, -1, b"k_exp"), ("v_exp", -65, -1, b"v_exp")])
def test_bad_4_bit_pools_are_refused(B, field, val, status, msg):
    kv, L = _kv4(B, **{field: val}), B.lib()
    assert L.bd_paged4_workspace_bytes(kv, 1, 1, 1) == 0
    for st in (_attend4(B, kv, _batch(B)), _append4(B, kv, _batch(B))):
        assert st == status and msg in L.bd_last_error()


def test_4_bit_exponents_of_fp16_rows(B):
    for e, ok in ((4, True), (5, False), (-14, True), (-15, False)):
        n = B.lib().bd_paged4_workspace_bytes(_kv4(B, dtype=B.F16, v_exp=e), 1, 1, 1)
        assert (n > 0) == ok


@pytest.mark.parametrize("field,val,msg", [
    ("n_requests", 0, b"n_requests"), ("table_width", 0, b"max_len"), ("max_len", 129, b"max_len"), ("page_table", None, b"page_table"),
    ("seq_len", 0x51002, b"seq_len"), ("row_start", None, b"row_start"), ("n_rows", -1, b"n_rows"), ("max_rows", 5, b"max_rows")])
def test_bad_batches_are_refused(B, field, val, msg):
    for st in (_attend4(B, _kv4(B), _batch(B, **{field: val})), _append4(B, _kv4(B), _batch(B, **{field: val}))):
        assert st == -1 and msg in B.lib().bd_last_error()


def test_bad_4_bit_attention_arguments_are_refused(B):
    L, kv, bt = B.lib(), _kv4(B), _batch(B)
    for kw, st, msg in ((dict(q=None), -1, b"q must"), (dict(qs=1028), -1, b"q must"), (dict(qs=1016), -1, b"q must"),
                        (dict(out=None), -1, b"out must"), (dict(out=0x60010), -1, b"overlap"), (dict(lse=0x90002), -1, b"lse"),
                        (dict(window=-1), -1, b"window"), (dict(sink=-1), -1, b"n_sink"), (dict(scale=0.0), -1, b"scale"),
                        (dict(scale=float("nan")), -1, b"scale"), (dict(ws=None), -5, b"workspace"), (dict(ws=0x100010), -5, b"workspace"),
                        (dict(n=0), -5, b"workspace")):
        assert _attend4(B, kv, bt, **kw) == st and msg in L.bd_last_error(), kw
    many = _batch(B, n_rows=40, max_rows=33)      # 132 rows of a KV head read a copy, which grows with the slots
    need = L.bd_paged4_workspace_bytes(kv, 2, 33, 100)
    assert _attend4(B, kv, many, n=need - 1) == -5
    assert L.bd_paged4_workspace_bytes(kv, 2, 33, 1000) > need > L.bd_paged4_workspace_bytes(kv, 2, 1, 100)
    assert L.bd_paged4_workspace_bytes(kv, 0, 1, 1) == 0 and L.bd_paged4_workspace_bytes(kv, 1, 1, -1) == 0
    assert _attend4(B, kv, _batch(B, n_rows=0, max_rows=0), q=None, out=None) == 0   # nothing to do


def test_bad_4_bit_append_arguments_are_refused(B):
    L, bt = B.lib(), _batch(B)
    for kw, msg in ((dict(k=None), b"k_new"), (dict(ks=248), b"k_new"), (dict(v=0x70008), b"v_new"), (dict(kh=0x68008), b"aligned"),
                    (dict(kh=0x60000, ks=264), b"not its own"), (dict(kh=0x70010), b"not its own"), (dict(vh=0x60000), b"not its own"),
                    (dict(kh=0x68000, vh=0x68010), b"overlap")):
        assert _append4(B, _kv4(B), bt, **kw) == -1 and msg in L.bd_last_error(), kw
    for kv in (_kv4(B, v=0x10000), _kv4(B, v=0x10030), _kv4(B, v_scale=0x30000), _kv4(B, k_scale=0x10008)):
        assert _append4(B, kv, bt) == -1 and b"overlap" in L.bd_last_error()


def _heads(B, n=4, pos=0x10000, q=0x20000, qs=1024, k=0x40000, ks=256, qo=0x60000, qos=1024, ko=0x80000, kos=256, **kw):
    c = B.HeadRope(B.BF16, 128, 128, 0, 8, 2, 1e-6, 0x90000, 0x90100, 0x91000)
    for key, v in kw.items():
        setattr(c, key, v)
    return B.lib().bd_head_norm_rope(c, n, pos, q, qs, k, ks, qo, qos, ko, kos, None)


@pytest.mark.parametrize("kw,st,msg", [
    (dict(dtype=1), -2, b"dtype"), (dict(head_dim=96), -2, b"head_dim"), (dict(rotary_dim=-16), -2, b"rotary_dim"), (dict(rotary_dim=24), -2, b"rotary_dim"),
    (dict(rotary_dim=144), -2, b"rotary_dim"), (dict(n_q_heads=-1), -1, b"head counts"), (dict(eps=0.0), -1, b"eps"), (dict(eps=float("nan")), -1, b"eps"),
    (dict(q_gain=0x90008), -1, b"gains"), (dict(turns=0x91004), -1, b"turns"), (dict(turns=None), -1, b"turns"), (dict(n=-1), -1, b"n_rows"),
    (dict(pos=None), -1, b"pos"), (dict(q=None), -1, b"q must"), (dict(k=0x40008), -1, b"k must"), (dict(qs=1016), -1, b"q must"),
    (dict(qos=1028), -1, b"q_out must"), (dict(ko=None), -1, b"k_out must"), (dict(qo=0x20010), -1, b"overlap"), (dict(qo=0x20000, qos=2048), -1, b"overlap"),
    (dict(ko=0x20000), -1, b"overlap"), (dict(qo=0x80000), -1, b"overlap"), (dict(qo=0x90010), -1, b"gain"), (dict(ko=0x10000), -1, b"pos or turns"),
    # rows of one projection side by side: keys right behind the queries are fine, over them not
    (dict(q=0x20000, qo=0x20000, qs=1536, qos=1536, k=0x20000 + 2032, ko=0x20000 + 2032, ks=1536, kos=1536), -1, b"overlap")])
def test_bad_head_norms_are_refused(B, kw, st, msg):
    assert _heads(B, **kw) == st and msg in B.lib().bd_last_error()


def test_head_norms_with_nothing_to_do(B):
    assert _heads(B, n=0, pos=None, q=None) == 0 and _heads(B, n_q_heads=0, n_kv_heads=0, q=None, k=None) == 0


def _logprobs(B, x=0x100000, stride=1000, dtype=1, rows=4, vocab=1000, temperature=1.0, tokens=0x10000, n=2, lp=0x11000, ent=0x12000, lse=0x13000, k=5,
              ids=0x14000, alt=0x15000):
    return B.lib().bd_token_logprobs(x, stride, dtype, rows, vocab, temperature, tokens, n, lp, ent, lse, k, ids, alt, None)


@pytest.mark.parametrize("kw,st,msg", [
    (dict(dtype=7), -2, b"dtype"), (dict(rows=-1), -1, b"rows"), (dict(vocab=0), -1, b"vocab"), (dict(n=65), -1, b"n_given"), (dict(k=33), -1, b"top_k"),
    (dict(vocab=3, stride=3, k=4), -1, b"at most vocab"), (dict(temperature=0.0), -1, b"temperature"), (dict(temperature=-1.0), -1, b"temperature"),
    (dict(temperature=float("nan")), -1, b"temperature"), (dict(temperature=float("inf")), -1, b"temperature"), (dict(temperature=1e-40), -1, b"temperature"),
    (dict(x=None), -1, b"logits"), (dict(x=0x100002), -1, b"logits"), (dict(stride=999), -1, b"logits"), (dict(tokens=None), -1, b"tokens"),
    (dict(lp=None), -1, b"logprob"), (dict(ids=None), -1, b"top_ids"), (dict(ent=0x12002), -1, b"entropy"), (dict(ent=0x100100), -1, b"overlap"),
    (dict(lse=0x12004), -1, b"overlap"), (dict(lp=0x10010), -1, b"overlap"), (dict(alt=0x14010), -1, b"overlap")])
def test_bad_logprobs_are_refused(B, kw, st, msg):
    assert _logprobs(B, **kw) == st and msg in B.lib().bd_last_error()


def test_logprobs_of_no_rows(B):
    assert _logprobs(B, rows=0, x=None, tokens=None) == 0


def test_python_checks_come_before_the_device(B):
    from block_drafter_gb300.paged import PagedCache4, PageTables
    from block_drafter_gb300.target import HeadNormRope, token_logprobs
    bf = torch.bfloat16
    c, s = torch.zeros(4, 2, 16, 32, dtype=torch.uint8), torch.zeros(4, 2, 16, 4, dtype=torch.uint8)
    for args, msg in (((c, s, c.clone(), s.clone()), "CUDA"), ((c, s, c[:3], s), "one shape"), ((c.float(), s, c.float(), s), "not supported"),
                      ((c, s[..., :2], c, s[..., :2]), "D/16"), ((c.permute(0, 1, 3, 2),) * 1 + (s, c.permute(0, 1, 3, 2), s), "contiguous")):
        with pytest.raises(ValueError, match=msg):
            PagedCache4(*args, n_q_heads=4, dtype=bf)
    with pytest.raises(ValueError, match="rows of"):
        PagedCache4(c, s, c.clone(), s.clone(), n_q_heads=4, dtype=torch.float32)
    with pytest.raises(B.BdError, match="multiple"):
        PagedCache4(c, s, c.clone(), s.clone(), n_q_heads=3, dtype=bf)
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        PageTables(i(3, 4), i(3), i(9), i(1), 16)
    with pytest.raises(ValueError, match="q_gain"):
        HeadNormRope(128, None, torch.ones(64, dtype=bf), None)
    with pytest.raises(ValueError, match="CUDA"):
        HeadNormRope(128, None, torch.ones(128, dtype=bf), None)
    with pytest.raises(ValueError, match="dtype"):
        HeadNormRope(128, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        HeadNormRope(128, None, None, None, dtype=bf)(torch.zeros(2, 3, 128, dtype=bf), None, i(2))
    with pytest.raises(ValueError, match="CUDA"):
        token_logprobs(torch.zeros(2, 9), i(2), torch.zeros(2))
    with pytest.raises(ValueError, match="logits"):
        token_logprobs(torch.zeros(2, 9).double(), i(2), torch.zeros(2))


def test_turns_are_the_angles():
    from block_drafter_gb300.target import turns_of
    import math
    f = torch.tensor([1.0, 0.0, math.pi / 2, 1e-7, 3.0, 7.0, -1.0], dtype=torch.float64)
    got = [t / 2.0 ** 64 for t in turns_of(f).tolist()]
    for g, w in zip(got, f.tolist()):
        assert abs((g - w / (2 * math.pi) + 0.5) % 1.0 - 0.5) < 2.0 ** -50
    assert turns_of(torch.tensor([2 * math.pi / 4], dtype=torch.float64)).tolist()[0] % 2 ** 64 != 2 ** 62   # fp64's pi / 2, not pi / 2
