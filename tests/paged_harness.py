"""Paged-cache cases for the GPU tests: pools with garbage wherever no request holds a slot,
ragged requests, guard rows, and tolerances from the roundings the kernels make."""
import dataclasses

import numpy as np
import torch

from oracle import paged_oracle as P

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@dataclasses.dataclass
class PagedCase:
    lens: tuple
    rows: tuple
    hkv: int = 2
    group: int = 4
    d: int = 128
    page: int = 16
    dtype: str = "bf16"
    window: int = 0
    n_sink: int = 0
    nhd: bool = False        # pool [pages, page size, KV heads, D] instead of [pages, KV heads, ...]
    pad: int = 0             # extra elements in every row stride and between pool slots
    lead: int = 0            # rows before the first request and behind the last one
    std: float = 1.0         # of the queries
    spare: int = 0           # entries beyond the longest request's in a page-table row
    seed: int = 0

    def build(self):
        from block_drafter_gb300.paged import PagedCache
        g = torch.Generator().manual_seed(self.seed * 7919 + sum(self.lens) * 31 + sum(self.rows))
        t, B, hq = TYPES[self.dtype], len(self.lens), self.hkv * self.group
        held = [-(-n // self.page) for n in self.lens]
        width, total = max(max(held), 1) + self.spare, sum(held) + 2
        ids = torch.randperm(total, generator=g)
        table = torch.full((B, width), 2 ** 30, dtype=torch.int32)  # entries behind a length are never followed
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = ids[at:at + h].int()
            at += h
        self.k, self.v = [], []  # fp64 contents in slot order
        D = self.d + self.pad
        shape = (total, self.page, self.hkv, D) if self.nhd else (total, self.hkv, self.page, D)
        pools = [torch.full(shape, float("nan"), dtype=t) for _ in range(2)]
        views = [(p.permute(0, 2, 1, 3) if self.nhd else p)[..., :self.d] for p in pools]
        for b, n in enumerate(self.lens):
            for pool, keep in zip(views, (self.k, self.v)):
                x = torch.randn(n, self.hkv, self.d, generator=g).to(t)
                j = torch.arange(n)
                pool[table[b, j // self.page].long(), :, j % self.page] = x
                keep.append(x.double().numpy())
        starts = [self.lead]
        for r in self.rows:
            starts.append(starts[-1] + r)
        self.starts, self.n_rows = starts, starts[-1] + self.lead
        q = torch.randn(self.n_rows, hq, self.d, generator=g) * self.std
        self.q = q.to(t)
        self.qf = self.q.double().numpy()
        self.scale = self.d ** -0.5
        cu = lambda x: x.cuda()
        dev = [cu(p) for p in pools]
        dv = [(p.permute(0, 2, 1, 3) if self.nhd else p)[..., :self.d] for p in dev]
        self.kd, self.vd = dv
        self.cache = PagedCache(dv[0], dv[1], n_q_heads=hq)
        self.table, self.lend = cu(table), cu(torch.tensor(self.lens, dtype=torch.int32))
        self.startd = cu(torch.tensor(starts, dtype=torch.int32))
        self.max_len, self.max_rows = max(self.lens), max(self.rows)
        self.batch = self.cache.batch(self.table, self.lend, self.startd, self.n_rows, self.max_rows, self.max_len)
        self.qd = self.strided(self.q)
        return self

    def strided(self, x):
        """x [rows, heads, D] on the GPU, its rows `pad` (rounded to 8) elements further apart."""
        rows, heads, d = x.shape
        wide = torch.full((rows, heads * d + 8 * self.pad), float("nan"), dtype=x.dtype, device="cuda")
        wide[:, :heads * d] = x.reshape(rows, heads * d).cuda()
        return wide[:, :heads * d].unflatten(1, (heads, d))

    def outputs(self):
        out = self.strided(torch.full((self.n_rows, self.hkv * self.group, self.d), -7.0, dtype=TYPES[self.dtype]))
        lse = torch.full((self.n_rows, self.hkv * self.group), -7.0, device="cuda")
        return out, lse

    def attend(self, **kw):
        out, lse = self.outputs()
        self.cache.attention(self.batch, self.qd, out, lse=lse, window=self.window, n_sink=self.n_sink, **kw)
        return out, lse

    def check_attention(self, out, lse, requests=None):
        """Against the oracle.  With p_j the weights of a row, A = sum_j p_j |v_j| and
        S = max_j scale |q|.|k_j|:
          * scores: D products and sums in fp32, truncated or rounded, are off by at most
            D 2^-23 S, and forming s log2(e) and 2^x by another (|s| + 4) 2^-22 <= (S + 4) 2^-22:
            ds; weights (numerator and sum) by a relative 2 ds (1.01 covers the exponential's
            second order, ds < 1e-2);
          * weights as a 16-bit operand of the second product: half a step u of the type;
          * sums in fp32 over n slots, and the joining of parts: (n + 64) 2^-23 A;
          * the output: half a step of the type, and of its smallest subnormal."""
        half = torch.finfo(TYPES[self.dtype]).eps / 2
        tiny = torch.finfo(TYPES[self.dtype]).smallest_normal * torch.finfo(TYPES[self.dtype]).eps / 2
        got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b, (n, r) in enumerate(zip(self.lens, self.rows)):
            if requests is not None and b not in requests:
                continue
            s = slice(self.starts[b], self.starts[b] + r)
            ref, rl, spread, size = P.attention(self.qf[s], self.k[b], self.v[b], self.window, self.n_sink, self.scale)
            ds = (self.d * 2.0 ** -23) * size + (size + 4) * 2.0 ** -22
            tol = half * np.abs(ref) + tiny + (half + 2.02 * ds[..., None] + (n + 64) * 2.0 ** -23) * spread
            empty = np.isinf(rl)
            assert (np.isneginf(glse[s]) == empty).all(), f"request {b}: rows without a visible slot"
            err = np.abs(got[s] - ref) - tol
            assert (err <= 0).all(), f"request {b}: worst {err.max()} beyond {tol.max()}"
            ltol = ds + (n + 64) * 2.0 ** -23 + np.abs(rl) * 2.0 ** -22
            lerr = np.abs(glse[s][~empty] - rl[~empty]) - ltol[~empty]
            assert (lerr <= 0).all(), f"request {b}: lse {lerr.max()}"

    def check_guards(self, out, lse):
        for t in (out, lse):
            for s in (slice(0, self.lead), slice(self.starts[-1], self.n_rows)):
                assert (t[s] == -7.0).all(), "rows outside every request changed"
