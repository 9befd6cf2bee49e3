"""GPU: attention over the cache where the weights of the visible keys, or the E4M3 scales of the keys, lie far
apart: many small weights beside a large one; keys a row does not see, or gives no weight, of any size.

The bound of tests/paged.py allows 2^-25 of sum |v|, what P in fp16 loses when its largest is 1, and of keys that
all rows see.  Here the kernels are held to what they promise: weights keep the 16-bit type's own bits down to
far below the row's largest.  For each row, with p the true weights (they sum to 1), v_j = code_j * 2^e_j (e_j = 0 in
a 16-bit cache) and sums over the visible keys only,

    |dO| <= (u + 2 ds) sum p |v| + u (1 + u) |O| + w max_j(p_j 2^e_j) sum_j |code_j| + 2^-126 (1 + max(p) sum |v|),

u half a step of the 16-bit type, ds = 2^-16 (R + 1) the scores' error as there.  The third term: in a 16-bit cache
P's largest is 2^15, and below 2^-14 fp16 is off by 2^-25, so w = 2^-40.  E4M3 weights p_j 2^e_j have a largest of
2^11 at least, which gives 2^-36; 128 keys whose scales are all within 2^8 may share a reference, which then
lies up to 2^8 above the row's own largest: w = 2^-28.  The last term is fp32's range: a weight below 2^-126 of the largest,
exp(-87.3), is zero where 32-bit sums of parts of the keys are merged (the factor 2^(m_i - m) of a part underflows), so
the key is lost with p |v| <= 2^-126 max(p) |v|; a result below fp16's normal range is off by 2^-25 itself."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_attention_111_b200 as fa
from tests.parity import ensure_built

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def exact(q, k, v, see, scale, e=None):
    """fp64 on the GPU: q [T, Hq, d], k, v [Hk, n, d], see [T, n], e [Hk, n].  O, LSE, sum p |v|, the third and the
    last term's max times sum, and R."""
    T, Hq, d = q.shape
    G = Hq // k.shape[0]
    q = q.double()
    o, a, low, tiny = (torch.zeros_like(q) for _ in range(4))
    lse, r = (torch.zeros(T, Hq, dtype=torch.float64, device=q.device) for _ in range(2))
    for h in range(Hq):
        kk, vv = k[h // G].double(), v[h // G].double()
        size = torch.ones_like(vv[:, 0]) if e is None else torch.exp2(e[h // G].double())
        for t in range(T):                               # visible keys only: the others may hold anything
            i = see[t].nonzero()[:, 0]
            s = scale * (kk[i] @ q[t, h])
            lse[t, h] = torch.logsumexp(s, 0)
            p = torch.exp(s - lse[t, h])
            o[t, h], a[t, h] = p @ vv[i], p @ vv[i].abs()
            low[t, h] = (p * size[i]).max() * (vv[i].abs() / size[i][:, None]).sum(0)
            tiny[t, h] = 1 + p.max() * vv[i].abs().sum(0)
            r[t, h] = (scale * (kk[i].abs() @ q[t, h].abs())).max()
    return o, lse, a, low, tiny, r


def check(q, o, lse, want, w=2.0 ** -40, label="", rows=None):
    u = float(torch.finfo(q.dtype).eps) / 2
    rows = slice(None) if rows is None else rows
    o, lse = o[rows], lse[rows]
    ro, rl, a, low, tiny, r = (x[rows] for x in want)
    ds = 2.0 ** -16 * (r + 1)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all(), f"{label}: not finite"
    dl = (lse.double() - rl).abs() - (ds + 2.0 ** -20 * (1 + rl.abs()))
    assert float(dl.max()) <= 0, f"{label}: lse over its bound by {float(dl.max())}"
    d = (o.double() - ro).abs()
    bound = (u + 2 * ds[..., None]) * a + u * (1 + u) * ro.abs() + w * low + 2.0 ** -126 * tiny
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
    check(q, o, lse, exact(q, *(x.view(1, -1, d)[:, :N + n] for x in (k, v)), see, d ** -0.5), label=f"2^-{down}")


class Filled:
    """An E4M3 cache of one sequence, written from k, v [N, Hk, d]; what it holds in fp64."""

    def __init__(self, k, v, page=16):
        ensure_built()
        N, Hk, d = k.shape
        pages = -(-N // page)
        g = torch.Generator().manual_seed(N)
        order = torch.randperm(pages, generator=g).to(device="cuda", dtype=torch.int32)
        codes = [torch.full((pages, Hk, page, d), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.full((pages, Hk, page), 200, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.cache = fa.KVCache(*codes, order[None].contiguous(), *scales)
        i32 = dict(dtype=torch.int32, device="cuda")
        fa.cache_append(self.cache, k.to(BF).cuda(), v.to(BF).cuda(), torch.tensor([0, N], **i32), torch.zeros(1, **i32))
        at = order.long()

        def dense(x):
            return x[at].transpose(0, 1).flatten(1, 2)[:, :N]

        self.k, self.v = (dense(c.view(torch.float8_e4m3fn)).double() * torch.exp2(dense(s).double() - 127)[..., None]
                          for c, s in zip(codes, scales))
        self.e = dense(scales[1]).double() - 127
        self.N, self.d = N, d

    def attend(self, q, n, mask=None, unseen=()):
        """The last n tokens attend: checks the rows that see none of the new tokens `unseen`."""
        i32 = dict(dtype=torch.int32, device="cuda")
        L = self.N - n
        o, lse = fa.attention_forward_tree(q, self.cache, torch.tensor([0, n], **i32), torch.tensor([L], **i32), n,
                                           tree_mask=mask)
        fa.fa_check_status()
        see = torch.ones(n, self.N, dtype=torch.bool, device="cuda")
        j = torch.arange(n, device="cuda")
        see[:, L:] = j[None] <= j[:, None] if mask is None else (mask[:, :1] >> j[None] & 1).bool()
        rows = ~see[:, [L + t for t in unseen]].any(1)
        assert rows.any()
        check(q, o, lse, exact(q, self.k, self.v, see, self.d ** -0.5, self.e), 2.0 ** -28, rows=rows)


def _rows(N, seed, heads=2, d=64):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(N, heads, d, generator=g)


@pytest.mark.parametrize("n", [2, 8, 40])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("which,up", [("v", 12), ("v", 24), ("v", 34), ("v", 60), ("v", 120), ("k", 17), ("k", 25), ("k", 40),
                                      ("k", 60), ("k", 120), ("kv", 30), ("kv", -40)])
def test_finite_keys_a_row_does_not_see_do_not_reach_it(which, up, dtype, tree, n):
    """Later tokens of a chain and siblings of a tree whose rows are 2^up times as large."""
    N = 200 + n
    k, v = _rows(N, 1), _rows(N, 2)
    big = [n - 1] if n < 20 else [n - 1, 20]
    for t in big:
        for x in ([k] if "k" in which else []) + ([v] if "v" in which else []):
            x[200 + t] *= 2.0 ** up
    c = Filled(k, v)
    mask = None
    if tree:                                             # a star: siblings do not see one another
        mask = fa.tree_mask([-1] + [0] * (n - 1), torch.tensor([0, n], device="cuda"))
    c.attend(_rows(n, 3, 4).to(dtype).cuda(), n, mask, big)


@pytest.mark.parametrize("n", [1, 6, 40])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("up", [12, 24, 40, 60])
@pytest.mark.parametrize("where", [0, 130, 199])
def test_large_values_of_no_weight(dtype, n, up, where):
    """Keys that all rows see, of values 2^up times as large and weights some 2^-(up + 30) as large."""
    N = 200 + n
    k, v, q = _rows(N, 1), _rows(N, 2), _rows(n, 3, 4)
    q[..., 0], k[..., 0] = 8.0, 0.0
    k[where] = 0
    k[where, :, 0] = -(up + 30) * float(np.log(2))
    v[where] *= 2.0 ** up
    Filled(k, v).attend(q.to(dtype).cuda(), n)


@pytest.mark.parametrize("n", [1, 6, 40])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("up", [17, 25, 40, 100])
def test_large_keys_across_the_queries(dtype, n, up):
    """Keys that are 2^up times as large as the others in a column where the queries are zero."""
    N = 200 + n
    k, v, q = _rows(N, 1), _rows(N, 2), _rows(n, 3, 4)
    q[..., 5] = 0
    k[..., 5] = 0
    for where in (3, 131, 198):
        k[where] = 0
        k[where, :, 5] = 2.0 ** up
    Filled(k, v).attend(q.to(dtype).cuda(), n)


@pytest.mark.parametrize("n", [1, 6, 40])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("step", [-30, -9, 9, 30])
def test_values_that_grow_or_fall_along_the_keys(dtype, n, step):
    """Each 64 keys' values are 2^step times those before, and the queries weigh only one block: each in turn."""
    N = 320 + n
    k, v = _rows(N, 1), _rows(N, 2)
    q = _rows(n, 3, 4)
    for b in range(5):
        v[64 * b:64 * b + 64] *= 2.0 ** (step * (b - 2))
    v[320:] *= 2.0 ** (-3 * abs(step))
    for b in range(5):
        kb = k.clone()
        kb[..., 0], q[..., 0] = 0.0, 8.0
        kb[:, :, 0] = -100.0
        kb[64 * b:64 * b + 64, :, 0] = 0.0
        if dtype is HF and step * (b - 2) > 12:
            continue                                     # not a result that fp16 holds
        Filled(kb, v).attend(q.to(dtype).cuda(), n)


@pytest.mark.parametrize("n", [1, 6, 40])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("step", [-100, 100])
def test_values_far_apart_from_one_tile_to_the_next(dtype, n, step):
    """Tiles of 128 keys, alike inside, whose values are 2^step times those of the tile before."""
    N = 384 + n
    k, v, q = _rows(N, 1), _rows(N, 2), _rows(n, 3, 4)
    for b in range(3):
        v[128 * b:128 * b + 128] *= 2.0 ** (step * (b - 1))
    v[384:] = 0
    k[..., 0], q[..., 0] = -100.0, 8.0
    for b in range(3):
        if dtype is HF and step * (b - 1) > 0:
            continue                                     # not a result that fp16 holds
        kb = k.clone()
        kb[128 * b:128 * b + 128, :, 0] = 0.0
        Filled(kb, v).attend(q.to(dtype).cuda(), n)


@pytest.mark.parametrize("n", [8, 40])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("N0", [0, 120, 200])
def test_unseen_keys_of_any_size_beside_some_that_are_not_finite(N0, dtype, n):
    """Siblings whose rows are NaN, infinite or 2^60 as large, in one tile."""
    N = N0 + n
    k, v = _rows(N, 1), _rows(N, 2)
    odd = [1, 2, 4, 5, 6]
    v[N0 + 1] = float("nan")
    v[N0 + 2] *= 2.0 ** 60
    k[N0 + 4] *= 2.0 ** 60
    k[N0 + 5, :, ::3] = float("nan")
    v[N0 + 6, :, 7] = float("inf")
    mask = fa.tree_mask([-1] + [0] * (n - 1), torch.tensor([0, n], device="cuda"))
    Filled(k, v).attend(_rows(n, 3, 4).to(dtype).cuda(), n, mask, odd)
