"""Shared helpers of the paged-cache tests: seeded caches with ragged lengths, and the error bound
of the attention over them."""

from __future__ import annotations

import numpy as np
import torch

import exact_attention_111_b200 as fa
import oracle.paged as ora
from tests.parity import ensure_built

TOP = {torch.bfloat16: 240.0 * 2.0 ** 120, torch.float16: 61440.0}


class Case:
    """A cache of B sequences: every slot that holds no token yet is garbage (NaN, or random codes)."""

    def __init__(self, lens, counts, Hk, d, page, dtype, fp8, seed, device="cuda", spare=3, k_gain=1.0):
        ensure_built()
        g = torch.Generator().manual_seed(seed)
        self.lens_l, self.counts_l, self.Hk, self.d, self.page, self.dtype, self.fp8 = (
            list(lens), list(counts), Hk, d, page, dtype, fp8)
        self.B = len(self.lens_l)
        need = [-(-(a + b) // page) for a, b in zip(lens, counts)]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        width = max(need + [1]) + 1
        table = np.full((self.B, width), -1, dtype=np.int32)      # unused entries are no pages
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table_np = table
        shape = (self.pages, Hk, page, d)
        self.total = sum(counts)
        self.cu_l = [sum(counts[:i]) for i in range(self.B + 1)]
        self.t = {}
        for n in ("k", "v"):
            x = torch.randn(shape, generator=g) * (k_gain if n == "k" else 1.0)
            if fp8:
                self.t[n] = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)   # NaN codes among them
                self.t[n + "_scale"] = torch.randint(0, 256, shape[:3], generator=g, dtype=torch.uint8)
                spread = torch.randint(119, 124, shape[:3], generator=g, dtype=torch.uint8)
                codes = (x * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                self.t[n] = torch.full(shape, float("nan"), dtype=dtype)
            for b in range(self.B):
                for p in range(lens[b]):
                    i, r = ora.slot(table, b, p, page)
                    if fp8:
                        self.t[n][i, :, r] = codes[i, :, r]
                        self.t[n + "_scale"][i, :, r] = spread[i, :, r]
                    else:
                        self.t[n][i, :, r] = x[i, :, r].to(dtype)
        self.g = g
        self.device = device
        self.gpu = {n: x.to(device) for n, x in self.t.items()}
        self.table = torch.from_numpy(table).to(device)
        self.lens = torch.tensor(self.lens_l, dtype=torch.int32, device=device)
        self.cu = torch.tensor(self.cu_l, dtype=torch.int32, device=device)
        self.cache = fa.KVCache(self.gpu["k"], self.gpu["v"], self.table, self.gpu.get("k_scale"),
                                self.gpu.get("v_scale"))

    def new(self, heads, pad=0):
        """[total + pad, heads, d] new rows."""
        return torch.randn(self.total + pad, heads, self.d, generator=self.g).to(self.dtype)

    def values(self):
        """(K, V) as the GPU's cache holds them now, fp64 numpy [pages, Hk, page, d]."""
        out = []
        for n in ("k", "v"):
            if self.fp8:
                s = self.gpu[n + "_scale"].cpu().numpy().astype(np.float64)
                with np.errstate(invalid="ignore", over="ignore"):
                    out.append(ora.e4m3_values(self.gpu[n].cpu().view(torch.uint8).numpy())
                               * np.exp2(s - 127)[..., None])
            else:
                out.append(self.gpu[n].cpu().double().numpy())
        return out

    def put(self, k_new, v_new):
        fa.cache_append(self.cache, k_new.to(self.device), v_new.to(self.device), self.cu, self.lens)


def check_attention(case, q, o, lse, scale, bits=None, label="", nan_ok=False):
    """Compare with fp64.  Per row: the scores are off by at most ds = 2^-16 (R + 1) (d <= 128
    fp32 accumulations of steps 2^-23 of R = max sum |q k|, the exponential's and the running
    max's rounding), so p by a factor 1 +- 2 ds (the sum's own error included);
    P is rounded to 16 bits (u relative, in fp16 2^-25 absolute below its normal range) and
    the result once more:   |dO| <= (u + 2 ds) sum p |v| + 2^-25 sum |v| + u |O| (+ 2^-25)."""
    u = float(torch.finfo(q.dtype).eps) / 2
    K, V = case.values()
    qd, od, ld = q.cpu().double().numpy(), o.cpu().double().numpy(), lse.cpu().double().numpy()
    bits = None if bits is None else bits.cpu().numpy().astype(np.uint64)
    for b in range(case.B):
        a, e = case.cu_l[b], case.cu_l[b + 1]
        if a == e:
            continue
        n = case.lens_l[b] + e - a
        k, v = ora.gather(K, case.table_np, b, n, case.page), ora.gather(V, case.table_np, b, n, case.page)
        ro, rl, A, W, R = ora.attend(qd[a:e], k, v, case.lens_l[b], scale, None if bits is None else bits[a:e])
        ds = 2.0 ** -16 * (R + 1)
        empty = np.isneginf(rl)
        assert np.array_equal(empty, np.isneginf(ld[a:e])), f"{label} b={b}: rows without keys"
        assert np.array_equal(np.isnan(rl), np.isnan(ld[a:e])), f"{label} b={b}: NaN rows"
        fine = np.isfinite(rl)
        dl = np.abs(np.where(fine, ld[a:e] - np.where(fine, rl, 0), 0))
        # the sum of at most 2^20 terms adds its own rounding, and the LSE its last one
        assert np.all(dl <= np.where(fine, ds + 2.0 ** -20 * (1 + np.abs(np.where(fine, rl, 0))), 0)), f"{label} b={b}: lse {dl.max()}"
        bad = ~np.isfinite(ro)
        if nan_ok:
            assert np.array_equal(bad, ~np.isfinite(od[a:e])), f"{label} b={b}: where it is finite"
            assert np.array_equal(np.isnan(ro), np.isnan(od[a:e])), f"{label} b={b}: NaN places"
            assert np.array_equal(ro[bad & ~np.isnan(ro)], od[a:e][bad & ~np.isnan(ro)]), f"{label} b={b}: infinities"
        else:
            assert not bad.any() and np.isfinite(od[a:e]).all(), f"{label} b={b}: not finite"
        ok = ~bad
        d = np.abs(np.where(ok, od[a:e], 0) - np.where(ok, ro, 0))
        bound = (u + 2 * ds[..., None]) * A + 2.0 ** -25 * (W + 1) + u * (1 + u) * np.abs(ro)
        worst = np.where(ok, d - np.where(ok, bound, 0), -1)
        assert np.all(worst <= 0), f"{label} b={b}: off by {d.max()} (over the bound by {worst.max()})"
        assert np.all(od[a:e][empty] == 0), f"{label} b={b}: rows without keys are zero"
