"""GPU: attention over the cache where the weights of the visible keys lie far apart: many small weights
beside a large one.

The bound of tests/paged.py allows 2^-25 of sum |v|, what P in fp16 loses when its largest is 1.  Here the
kernels are held to what they promise: weights keep the 16-bit type's own bits down to far below the
largest.  For each row, with p the true weights (they sum to 1) and sums over the visible keys only,

    |dO| <= (u + 2 ds) sum p |v| + u (1 + u) |O| + 2^-40 max(p) sum |v| + 2^-126,

u half a step of the 16-bit type, ds = 2^-16 (R + 1) the scores' error as there.  The third term: P's largest is
2^15, and below 2^-14 fp16 is off by 2^-25, 2^-40 of the largest.  The last term is what fp32 resolves;
a result below fp16's normal range is off by 2^-25 itself."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_attention_111_b200 as fa
from tests.parity import ensure_built

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def exact(q, k, v, see, scale):
    """fp64 on the GPU: q [T, Hq, d], k, v [Hk, n, d], see [T, n].  O, LSE, sum p |v|, max(p) sum |v| and R."""
    T, Hq, d = q.shape
    G = Hq // k.shape[0]
    q = q.double()
    o, a, low = (torch.zeros_like(q) for _ in range(3))
    lse, r = (torch.zeros(T, Hq, dtype=torch.float64, device=q.device) for _ in range(2))
    for h in range(Hq):
        kk, vv = k[h // G].double(), v[h // G].double()
        for t in range(T):                               # visible keys only: the others may hold anything
            i = see[t].nonzero()[:, 0]
            s = scale * (kk[i] @ q[t, h])
            lse[t, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[t, h])
            o[t, h], a[t, h], low[t, h] = p @ vv[i], p @ vv[i].abs(), p.max() * vv[i].abs().sum(0)
            r[t, h] = (scale * (kk[i].abs() @ q[t, h].abs())).max()
    return o, lse, a, low, r


def check(q, o, lse, want, label=""):
    u = float(torch.finfo(q.dtype).eps) / 2
    ro, rl, a, low, r = want
    ds = 2.0 ** -16 * (r + 1)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all(), f"{label}: not finite"
    dl = (lse.double() - rl).abs() - (ds + 2.0 ** -20 * (1 + rl.abs()))
    assert float(dl.max()) <= 0, f"{label}: lse over its bound by {float(dl.max())}"
    d = (o.double() - ro).abs()
    bound = (u + 2 * ds[..., None]) * a + u * (1 + u) * ro.abs() + 2.0 ** -40 * low + 2.0 ** -126
    bound = bound + (2.0 ** -25 if q.dtype is HF else 0.0)
    over = (d / bound).max()
    assert float(over) <= 1, f"{label}: {float(over)} times the bound (off by {float(d.max())})"


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("dtype", [HF, BF])
@pytest.mark.parametrize("down", [18, 24, 27])
def test_many_small_weights_beside_a_large_one(dtype, n, down):
    """One key in 32 is 2^(down - 0.5) times as heavy as each of the others, whose values are the larger ones: the
    small weights decide the result."""
    ensure_built()
    page, d, N = 128, 64, 20000
    pages = -(-(N + n) // page)
    g = torch.Generator(device="cuda").manual_seed(down)
    k = torch.zeros(pages, 1, page, d, device="cuda")
    v = (torch.rand(pages, 1, page, d, generator=g, device="cuda") + 0.5) * 2.0 ** 13
    k.view(-1, d)[7::32, 0] = 8.0
    v.view(-1, d)[7::32] *= 2.0 ** -19
    q = torch.zeros(n, 2, d, device="cuda")
    q[:, :, 0] = (down - 0.5) * float(np.log(2)) / (8.0 * d ** -0.5)
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    cache = fa.KVCache(k, v, torch.arange(pages, dtype=torch.int32, device="cuda")[None])
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [N]))
    o, lse = fa.attention_forward_tree(q, cache, cu, lens, n)
    fa.fa_check_status()
    see = torch.arange(N + n, device="cuda")[None] <= N + torch.arange(n, device="cuda")[:, None]
    check(q, o, lse, exact(q, *(x.view(1, -1, d)[:, :N + n] for x in (k, v)), see, d ** -0.5), f"2^-{down}")
