"""Paged cache without a GPU: the oracle's closed cases and the calls the library refuses."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P


@pytest.fixture(scope="module")
def B():
    from block_drafter_gb300 import builder
    builder.build()
    from block_drafter_gb300 import binding
    binding.lib()
    return binding


# ------------------------------------------------------------------ oracle
def test_visible_slots_by_hand():
    see = P.visible(6, 2, 3, 1)
    assert see.tolist() == [[True, False, True, True, True, False], [True, False, False, True, True, True]]
    assert P.visible(3, 5, 0, 0).sum(1).tolist() == [0, 0, 1, 2, 3]     # more rows than slots
    assert P.visible(4, 1, 1, 0).tolist() == [[False, False, False, True]]


def test_oracle_attention_of_one_slot_is_its_value_and_equal_keys_average():
    rng = np.random.default_rng(0)
    q, v = rng.normal(size=(1, 2, 4)), rng.normal(size=(3, 1, 4))
    k = np.repeat(rng.normal(size=(1, 1, 4)), 3, 0)
    out, lse, _, _ = P.attention(q, k, v, 0, 0, 0.5)
    np.testing.assert_allclose(out[0, 0], v[:, 0].mean(0))
    np.testing.assert_allclose(lse[0, 1], np.log(3) + 0.5 * k[0, 0] @ q[0, 1])
    out, _, _, _ = P.attention(q, k, v, 1, 0, 0.5)
    np.testing.assert_allclose(out[0, 1], v[2, 0])


def test_oracle_weights_spread_one_per_row_and_head():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    _, lse, _, _ = P.attention(q, k, v, 4, 1, 0.3)
    w = P.weights(q, k, lse, 2, 4, 1, 0.3)
    np.testing.assert_allclose(w.sum(), 2 * 4)
    assert w[8] == 0                                     # only the third row sees the last slot


def test_oracle_eviction_by_hand():
    s = np.array([0.0, 5, 5, 9, np.nan, -np.inf, 5, 1])
    assert P.evict(s, 8, 5, 1, 1) == [0, 1, 2, 3, 7]     # ties: the lower slots
    assert P.evict(s, 8, 8, 1, 1) == list(range(8))
    assert P.evict(s, 8, 2, 1, 1) == [0, 7]
    assert P.evict(s, 8, 7, 0, 1) == [0, 1, 2, 3, 4, 6, 7]  # NaN counts as -inf: a tie with slot 5


# ------------------------------------------------------------------ refusals
def _kv(B, **kw):
    c = B.PagedKv(8, 2, 128, B.BF16, 16, 10, 2 * 16 * 128, 16 * 128, 128, 0x10000, 0x20000)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _batch(B, **kw):
    t = B.PagedBatch(2, 8, 4, 2, 100, 0x30000, 0x31000, 0x32000)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def _attend(B, kv, bt, q=0x40000, qs=1024, out=0x80000, os=1024, lse=None, window=0, sink=0, scale=0.1, ws=0x100000, n=1 << 30):
    return B.lib().bd_paged_attention(kv, bt, q, qs, out, os, lse, window, sink, scale, ws, n, None)


@pytest.mark.parametrize("field,val,status,msg", [
    ("dtype", 1, -2, b"dtype"), ("dtype", 7, -2, b"dtype"), ("head_dim", 96, -2, b"head_dim"),
    ("n_q_heads", 7, -1, b"multiple"), ("n_kv_heads", 0, -1, b"multiple"), ("n_q_heads", 258, -2, b"128 query heads"),
    ("page_size", 0, -1, b"page_size"), ("n_pages", 0, -1, b"n_pages"), ("k", None, -1, b"pools"),
    ("v", 0x20008, -1, b"aligned"), ("slot_stride", 132, -1, b"multiples of 8"), ("page_stride", -8, -1, b">= 0"),
    ("head_stride", 64, -1, b"at least head_dim"), ("slot_stride", 0, -1, b"at least head_dim")])
def test_bad_pools_are_refused(B, field, val, status, msg):
    kv, L = _kv(B, **{field: val}), B.lib()
    assert L.bd_paged_workspace_bytes(kv, 1, 1) == 0
    for st in (_attend(B, kv, _batch(B)),
               L.bd_paged_append(kv, _batch(B), 0x40000, 256, 0x50000, 256, None),
               L.bd_paged_weights(kv, _batch(B), 0x40000, 1024, 0x60000, None, 0, 0, 0.1, 1.0, None, 0x70000, 100, None),
               L.bd_paged_evict(kv, _batch(B), 0x70000, 100, 50, 1, 1, None, 0, 0x71000, 0x72000, None, 0, None)):
        assert st == status and msg in L.bd_last_error()


@pytest.mark.parametrize("field,val,msg", [
    ("n_requests", 0, b"n_requests"), ("n_requests", 1025, b"n_requests"), ("table_width", 0, b"max_len"),
    ("max_len", 129, b"max_len"), ("max_len", -1, b"max_len"), ("page_table", None, b"page_table"),
    ("seq_len", None, b"seq_len"), ("seq_len", 0x31002, b"seq_len"), ("row_start", None, b"row_start"),
    ("n_rows", -1, b"n_rows"), ("max_rows", 5, b"max_rows"), ("max_rows", -1, b"max_rows")])
def test_bad_batches_are_refused(B, field, val, msg):
    st = _attend(B, _kv(B), _batch(B, **{field: val}))
    assert st == -1 and msg in B.lib().bd_last_error()


def test_bad_attention_arguments_are_refused(B):
    L, kv, bt = B.lib(), _kv(B), _batch(B)
    nan, inf = float("nan"), float("inf")
    for kw, st, msg in ((dict(q=None), -1, b"q must"), (dict(q=0x40008), -1, b"q must"), (dict(qs=1028), -1, b"q must"),
                        (dict(qs=1016), -1, b"q must"), (dict(out=None), -1, b"out must"), (dict(out=0x40010), -1, b"overlap"),
                        (dict(lse=0x90002), -1, b"lse"), (dict(window=-1), -1, b"window"), (dict(sink=-1), -1, b"n_sink"),
                        (dict(scale=0.0), -1, b"scale"), (dict(scale=nan), -1, b"scale"), (dict(scale=inf), -1, b"scale"),
                        (dict(ws=None), -5, b"workspace"), (dict(ws=0x100010), -5, b"workspace"), (dict(n=0), -5, b"workspace")):
        assert _attend(B, kv, bt, **kw) == st and msg in L.bd_last_error(), kw
    assert L.bd_paged_workspace_bytes(kv, 0, 1) == 0 and L.bd_paged_workspace_bytes(kv, 1, -1) == 0
    assert _attend(B, kv, _batch(B, n_rows=0, max_rows=0), q=None, out=None) == 0   # nothing to do


def test_bad_append_weights_and_eviction_arguments_are_refused(B):
    L, kv, bt = B.lib(), _kv(B), _batch(B)
    for k, ks, v, vs, msg in ((None, 256, 0x50000, 256, b"k_new"), (0x40000, 248, 0x50000, 256, b"k_new"),
                              (0x40000, 256, 0x50008, 256, b"v_new"), (0x40000, 256, 0x50000, 257, b"v_new")):
        assert L.bd_paged_append(kv, bt, k, ks, v, vs, None) == -1 and msg in L.bd_last_error()

    def weights(q=0x40000, lse=0x60000, used=None, decay=1.0, sin=None, sout=0x70000, stride=100):
        return L.bd_paged_weights(kv, bt, q, 1024, lse, used, 0, 0, 0.1, decay, sin, sout, stride, None)
    for kw, msg in ((dict(lse=None), b"lse"), (dict(used=0x60002), b"rows_used"), (dict(decay=float("inf")), b"decay"),
                    (dict(sout=None), b"score_out"), (dict(stride=99), b"max_len"), (dict(sin=0x70100), b"overlap")):
        assert weights(**kw) == -1 and msg in L.bd_last_error(), kw

    def evict(score=0x70000, stride=100, budget=50, sink=1, recent=1, dst=None, width=0, kept=0x80000, n=0x90000, so=None, sos=0):
        return L.bd_paged_evict(kv, bt, score, stride, budget, sink, recent, dst, width, kept, n, so, sos, None)
    for kw, msg in ((dict(budget=0), b"budget"), (dict(sink=-1), b"budget"), (dict(sink=25, recent=26), b"budget"),
                    (dict(score=None), b"score"), (dict(stride=99), b"score"), (dict(kept=None), b"kept_out"),
                    (dict(n=None), b"len_out"), (dict(dst=0x33000, width=3), b"dst_table"), (dict(dst=0x30000, width=8), b"page_table"),
                    (dict(so=0x70010, sos=100), b"overlap"), (dict(so=0x70000, sos=99), b"same stride"), (dict(so=0xa0000, sos=49), b"score_out")):
        assert evict(**kw) == -1 and msg in L.bd_last_error(), kw


def test_an_evictions_outputs_do_not_overlap(B):
    L, kv, bt = B.lib(), _kv(B), _batch(B)               # 2 requests, seq_len at 0x31000; 400 bytes of scores each
    for kept, n, so, sos in ((0x80000, 0x31004, None, 0),            # the lengths, shifted
                             (0x80000, 0x30ffc, None, 0), (0x80000, 0x80000, None, 0), (0x80000, 0x8018c, None, 0),
                             (0x31000 - 396, 0x90000, None, 0),      # the last kept slot is the first length
                             (0x70100, 0x90000, None, 0), (0x80000, 0x70004, None, 0),
                             (0x80000, 0x90000, 0x80100, 50), (0x80000, 0xa0004, 0xa0000, 50)):
        assert L.bd_paged_evict(kv, bt, 0x70000, 100, 50, 1, 1, None, 0, kept, n, so, sos, None) == -1, hex(kept)
        assert b"overlap" in L.bd_last_error()


def test_pools_whose_slots_overlap_are_not_stored_to(B):
    L, bt = B.lib(), _batch(B)
    evict = lambda kv: L.bd_paged_evict(kv, bt, 0x70000, 100, 50, 1, 1, None, 0, 0x80000, 0x90000, None, 0, None)
    for off in (-240, -16, 16, 240):                     # a slot of 128 values: 256 bytes
        kv = _kv(B, v=0x10000 + off)
        for k, v in ((0x40000, 0x50000), (0x40000, 0x40000)):
            assert L.bd_paged_append(kv, bt, k, 256, v, 256, None) == -1 and b"one pool" in L.bd_last_error()
        assert evict(kv) == -1 and b"overlap" in L.bd_last_error()
    one = _kv(B, v=0x10000)                              # one pool takes one set of rows
    assert L.bd_paged_append(one, bt, 0x40000, 256, 0x50000, 256, None) == -1 and b"one pool" in L.bd_last_error()
    assert L.bd_paged_append(one, bt, 0x40000, 256, 0x40000, 264, None) == -1 and b"one pool" in L.bd_last_error()


def test_python_checks_come_before_the_device(B):
    from block_drafter_gb300.paged import PagedCache
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        PagedCache(k, k.clone(), n_q_heads=4)
    with pytest.raises(ValueError, match="one shape"):
        PagedCache(k, k[:3], n_q_heads=4)
    with pytest.raises(ValueError, match="contiguous"):
        PagedCache(k.permute(0, 1, 3, 2), k.permute(0, 1, 3, 2), n_q_heads=4)
    with pytest.raises(ValueError, match="not supported"):
        PagedCache(k.double(), k.double(), n_q_heads=4)
    with pytest.raises(B.BdError, match="multiple"):
        PagedCache(k, k.clone(), n_q_heads=3)
    f = k.float()
    with pytest.raises(B.BdError, match="dtype"):
        PagedCache(f, f.clone(), n_q_heads=4)


# ------------------------------------------------------------------ launch plans
_CLUSTERS = r'''
#include <cuda_runtime.h>
static int device = 0, asked = 0;
static bool fails = true;
extern "C" cudaError_t cudaGetDevice(int *d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(void (*)(int), cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int *n, void (*)(int), const cudaLaunchConfig_t *c) {
  ++asked;
  *n = (device ? 100 : 10) / static_cast<int>(c->gridDim.x);
  return fails ? cudaErrorUnknown : cudaSuccess;
}
#include "bd_paged.h"
static void kernel(int) {}
int main() {
  const bd::ClustersAtOnce fit(kernel, 128, 1024);
  if (fit.of(4) != 0) return 1;                    // no answer: no clusters
  fails = false;
  if (fit.of(4) != 2 || fit.of(2) != 5) return 2;  // asked again
  device = 1;
  if (fit.of(4) != 25 || fit.of(16) != 6) return 3;
  device = 0;
  const int before = asked;
  if (fit.of(4) != 2 || fit.of(2) != 5 || asked != before) return 4;  // kept
  return fit.of(1) < 1000;
}
'''


def _run_host_program(tmp_path, text):
    import os
    import subprocess
    from block_drafter_gb300 import builder
    src, exe = tmp_path / "host.cpp", tmp_path / "host"
    src.write_text(text)
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    p = subprocess.run(["g++", "-std=c++17", "-O1", f"-I{builder.CSRC}", f"-I{builder.INCLUDE}", f"-I{cuda}", str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    assert subprocess.run([str(exe)]).returncode == 0


def test_cluster_counts_are_each_devices_own_and_failed_questions_are_asked_again(tmp_path):
    _run_host_program(tmp_path, _CLUSTERS)


_WORDS = r'''
#include "bd_internal.h"
int main() {
  unsigned word = 0;
  int copies = 0;
  auto read = [&](unsigned &v) { ++copies; v = word; return true; };
  auto write = [&](unsigned v) { ++copies; word = v; };
  if (bd::take_if_set(read, write) != 0 || copies != 1) return 1;  // nothing set: one copy
  word = 6;
  if (bd::take_if_set(read, write) != 6 || word != 0 || copies != 3) return 2;
  word = 2;
  return bd::take_if_set([](unsigned &) { return false; }, write) != 0 || word != 2;  // not read: kept
}
'''


def test_a_status_call_copies_an_error_word_back_only_where_it_was_set(tmp_path):
    _run_host_program(tmp_path, _WORDS)
