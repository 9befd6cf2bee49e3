"""GPU: the variants that only large calls take: a prompt's append, units of the attention cut over most of the GPU, and
long sequences in every kernel."""

from __future__ import annotations

import pytest
import torch

import exact_attention_111_b200 as fa
from tests.parity import ensure_built
from tests.paged import TOP
from tests.test_gpu_tree_weights import check, exact

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
I32 = dict(dtype=torch.int32, device="cuda")


def _quantise(x, dtype):
    """Codes and scale codes of rows x, from the definition; all values finite."""
    x = x.double().clamp(-TOP[dtype], TOP[dtype])
    top = x.abs().amax(-1, keepdim=True)
    e = torch.full_like(top, -126.0)
    m, ex = torch.frexp(top)                             # top = m 2^ex, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(top > 0, torch.maximum(e, (ex - 9 + (m > 0.875).to(ex.dtype)).double()), e)
    y = (x * torch.exp2(-e)).float()                     # a 16-bit value times a power of two: exact
    return y.to(torch.float8_e4m3fn).view(torch.uint8), (e[..., 0] + 127).to(torch.uint8)


def _cache(lens, Hk, d, page, dtype, fp8, seed=0):
    """An empty cache with room for lens, its pages in random order: (cache, order of the pages by sequence)."""
    ensure_built()
    need = [-(-n // page) for n in lens]
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(sum(need), generator=g).to(device="cuda")
    table, at = torch.zeros(len(lens), max(need), **I32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (sum(need), Hk, page, d)
    if not fp8:
        return fa.KVCache(*(torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(2)), table)
    return fa.KVCache(*(torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)), table,
                      *(torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") for _ in range(2)))


def _held(cache, x, b, n):
    """Positions 0 .. n - 1 of sequence b of one of the cache's tensors: [n, Hk, ..]."""
    pos = torch.arange(n, device="cuda")
    return x[cache.page_table[b, pos // cache.page_size].long(), :, pos % cache.page_size]


@pytest.mark.parametrize("d,Hk,dtype,fp8", [(128, 4, BF, True), (128, 5, HF, True), (128, 11, BF, True), (128, 7, BF, False),
                                            (128, 16, HF, False), (64, 8, HF, True), (64, 9, BF, True), (64, 17, HF, True),
                                            (64, 17, BF, False), (64, 3, BF, True), (128, 3, HF, True)])
def test_prompts_are_appended(d, Hk, dtype, fp8):
    """Calls about the size from which a warp takes four groups of heads, on both sides of it, with key heads that do
    not fill the last group."""
    edge = -(-3 * 2 ** 22 // (Hk * d))                   # tokens
    g = torch.Generator(device="cuda").manual_seed(Hk)
    for total in (edge - 1, edge, edge + 777):
        counts = [total // 3, 0, total - total // 3]
        lens = [13, 5, 0]
        cache = _cache([a + b for a, b in zip(lens, counts)], Hk, d, 16, dtype, fp8)
        x = torch.randn(total, 2 * Hk + 1, d, generator=g, device="cuda")
        x *= torch.exp2(torch.randint(-6, 6, (total, 2 * Hk + 1, 1), generator=g, device="cuda"))
        x = x.to(dtype)
        kn, vn = x[:, :Hk], x[:, Hk + 1:]
        cu = torch.tensor([0, counts[0], counts[0], total], **I32)
        fa.cache_append(cache, kn, vn, cu, torch.tensor(lens, **I32))
        fa.fa_check_status()
        at = 0
        for b, n in enumerate(counts):
            for new, store, scale in ((kn, cache.k, cache.k_scale), (vn, cache.v, cache.v_scale)):
                new = new[at:at + n]
                want, ws = _quantise(new, dtype) if fp8 else (new, None)
                assert torch.equal(_held(cache, store, b, lens[b] + n)[lens[b]:], want)
                assert torch.all(_held(cache, store, b, lens[b]) == 0)
                if fp8:
                    assert torch.equal(_held(cache, scale, b, lens[b] + n)[lens[b]:], ws)
            at += n


@pytest.mark.parametrize("n,Hq", [(1, 1), (1, 8), (2, 8), (4, 8), (9, 4), (64, 2), (150, 2)])
@pytest.mark.parametrize("d,dtype,fp8", [(128, BF, False), (64, HF, False), (128, HF, True), (64, BF, True)])
def test_one_unit_over_the_whole_gpu(n, Hq, d, dtype, fp8):
    """One sequence, one key head: one unit, whose parts lie on all 148 CTAs, as many as a merge can have."""
    N = 38000
    cache = _cache([N + n], 1, d, 128, dtype, fp8, seed=n)
    g = torch.Generator(device="cuda").manual_seed(n + Hq)
    k, v = (torch.randn(N + n, 1, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    k[:: 5000] *= 2                                      # parts whose largest scores differ
    fa.cache_append(cache, k, v, torch.tensor([0, N + n], **I32), torch.zeros(1, **I32))
    q = torch.randn(n, Hq, d, generator=g, device="cuda").to(dtype)
    ws = torch.full((fa.fa_fwd_tree_workspace_bytes(n, Hq, 1, d) // 4,), float("nan"), device="cuda")
    o, lse = fa.attention_forward_tree(q, cache, torch.tensor([0, n], **I32), torch.tensor([N], **I32), n, workspace=ws)
    fa.fa_check_status()
    K, V = (_held(cache, x, 0, N + n).transpose(0, 1) for x in (cache.k, cache.v))
    e = None
    if fp8:
        ks, e = (_held(cache, x, 0, N + n).transpose(0, 1).double() - 127 for x in (cache.k_scale, cache.v_scale))
        K, V = (x.view(torch.float8_e4m3fn).double() * torch.exp2(s)[..., None] for x, s in ((K, ks), (V, e)))
    rows = sorted({0, n // 2, n - 1})                    # the rows that are checked
    see = torch.arange(N + n, device="cuda")[None] <= N + torch.tensor(rows, device="cuda")[:, None]
    check(q[rows], o[rows], lse[rows], exact(q[rows], K.double(), V.double(), see, d ** -0.5, e),
          2.0 ** -28 if fp8 else 2.0 ** -40, f"{n} tokens")


@pytest.mark.parametrize("n,page", [(40, 16), (100, 128)])
@pytest.mark.parametrize("d,dtype,fp8", [(128, BF, False), (64, HF, False), (128, HF, True), (64, BF, True)])
def test_long_ragged_sequences_of_many_rows(n, page, d, dtype, fp8):
    """Many-row units of thousands of keys, several to a CTA and cut between CTAs."""
    lens, counts, Hk, Hq = [9000, 3, 4200, 12001], [n, n - 7, 1, n // 2], 2, 6
    cache = _cache([a + b for a, b in zip(lens, counts)], Hk, d, page, dtype, fp8, seed=n)
    g = torch.Generator(device="cuda").manual_seed(n)
    ends = [a + b for a, b in zip(lens, counts)]
    k, v = (torch.randn(sum(ends), Hk, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    fa.cache_append(cache, k, v, torch.tensor([sum(ends[:i]) for i in range(5)], **I32), torch.zeros(4, **I32))
    q = torch.randn(sum(counts), Hq, d, generator=g, device="cuda").to(dtype)
    cu = [sum(counts[:i]) for i in range(5)]
    o, lse = fa.attention_forward_tree(q, cache, torch.tensor(cu, **I32), torch.tensor(lens, **I32), n)
    fa.fa_check_status()
    for b, N in enumerate(ends):
        K, V = (_held(cache, x, b, N).transpose(0, 1) for x in (cache.k, cache.v))
        e = None
        if fp8:
            ks, e = (_held(cache, x, b, N).transpose(0, 1).double() - 127 for x in (cache.k_scale, cache.v_scale))
            K, V = (x.view(torch.float8_e4m3fn).double() * torch.exp2(s)[..., None] for x, s in ((K, ks), (V, e)))
        t = sorted({0, counts[b] // 2, counts[b] - 1})
        rows = [cu[b] + i for i in t]
        see = torch.arange(N, device="cuda")[None] <= lens[b] + torch.tensor(t, device="cuda")[:, None]
        check(q[rows], o[rows], lse[rows], exact(q[rows], K.double(), V.double(), see, d ** -0.5, e),
              2.0 ** -28 if fp8 else 2.0 ** -40, f"sequence {b}")
