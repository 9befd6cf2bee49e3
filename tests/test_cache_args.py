"""CPU-only: argument checks of the paged-cache entry points (they come back before any CUDA call),
and the host arithmetic of the serving helpers."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_attention_111_b200 as fa
import oracle.paged as ora
from exact_attention_111_b200 import build as fabuild

FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    fabuild.build()
    return fa.lib()


def _cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, page_table=FAKE, pages=8, Hk=2, page_size=16, d=64,
             dtype=fa.FA_BF16, B=2, max_pages=4, table_stride=4)
    a.update(kw)
    return fa.CacheArgs(*[a[n] for n, _ in fa.CacheArgs._fields_])


def _call(L, which, cache=None, **kw):
    c = _cache(**(cache or {}))
    if which == "append":
        a = dict(k_new=FAKE, v_new=FAKE, k_token_stride=128, k_head_stride=64, v_token_stride=128, v_head_stride=64,
                 cu_new=FAKE, lens=FAKE, total=4, dtype=fa.FA_BF16, stream=None)
        cls, f = fa.CacheAppendArgs, L.fa_cache_append
    elif which == "read":
        a = dict(lens=FAKE, k_out=FAKE, v_out=FAKE, N=64, dtype=fa.FA_BF16, stream=None)
        cls, f = fa.CacheReadArgs, L.fa_cache_read
    elif which == "keep":
        a = dict(lens=FAKE, kept=FAKE, counts=FAKE, width=3, stream=None)
        cls, f = fa.CacheKeepArgs, L.fa_cache_keep
    else:
        a = dict(q=FAKE, o=FAKE, lse=FAKE, q_token_stride=256, q_head_stride=64, o_token_stride=256, o_head_stride=64,
                 cu_new=FAKE, lens=FAKE, tree_mask=None, mask_words=0, total=4, Hq=4, max_new=2, dtype=fa.FA_BF16,
                 scale=0.125, workspace=FAKE, workspace_bytes=fa.fa_fwd_tree_workspace_bytes(4, 4, 2, 64), stream=None)
        cls, f = fa.TreeArgs, L.fa_fwd_tree
    a.update(kw)
    return f(bytes(cls(c, *[a[n] for n, _ in cls._fields_[1:]])))


BAD_CACHE = [
    (dict(k=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"), (dict(page_table=None), "INVALID_ARG"),
    (dict(k=FAKE + 8), "INVALID_ARG"), (dict(page_table=FAKE + 2), "INVALID_ARG"),
    (dict(pages=0), "INVALID_ARG"), (dict(Hk=0), "INVALID_ARG"), (dict(B=0), "INVALID_ARG"),
    (dict(max_pages=0), "INVALID_ARG"), (dict(table_stride=3), "INVALID_ARG"),
    (dict(d=96), "UNSUPPORTED"), (dict(page_size=8), "UNSUPPORTED"), (dict(page_size=48), "UNSUPPORTED"),
    (dict(page_size=256), "UNSUPPORTED"), (dict(dtype=fa.FA_FP32), "UNSUPPORTED"), (dict(dtype=9), "UNSUPPORTED"),
    (dict(pages=2 ** 30, Hk=1), "UNSUPPORTED"), (dict(max_pages=2 ** 28, table_stride=2 ** 28), "UNSUPPORTED"),
    (dict(dtype=fa.FA_E4M3), "INVALID_ARG"),
    (dict(dtype=fa.FA_E4M3, k_scale=FAKE, v_scale=FAKE + 1), "INVALID_ARG"),
]


@pytest.mark.parametrize("which", ["append", "read", "keep", "tree"])
def test_cache_errors(L, which):
    for kw, code in BAD_CACHE:
        assert _call(L, which, cache=kw) == getattr(fa, "FA_ERR_" + code), (which, kw)
    for f in (L.fa_cache_append, L.fa_cache_read, L.fa_cache_keep, L.fa_fwd_tree):
        assert f(None) == fa.FA_ERR_INVALID_ARG


def test_append_errors(L):
    for kw, code in [(dict(k_new=None), "INVALID_ARG"), (dict(v_new=FAKE + 4), "INVALID_ARG"),
                     (dict(k_token_stride=100), "INVALID_ARG"), (dict(v_head_stride=-64), "INVALID_ARG"),
                     (dict(cu_new=None), "INVALID_ARG"), (dict(lens=None), "INVALID_ARG"), (dict(total=-1), "INVALID_ARG"),
                     (dict(dtype=fa.FA_FP16), "UNSUPPORTED"), (dict(dtype=fa.FA_E4M3), "UNSUPPORTED")]:
        assert _call(L, "append", **kw) == getattr(fa, "FA_ERR_" + code), kw
    assert _call(L, "append", total=0, k_new=None, v_new=None) == fa.FA_OK     # nothing to do


def test_read_and_keep_errors(L):
    for kw, code in [(dict(k_out=None), "INVALID_ARG"), (dict(v_out=FAKE + 8), "INVALID_ARG"), (dict(N=-1), "INVALID_ARG"),
                     (dict(lens=None), "INVALID_ARG"), (dict(dtype=fa.FA_FP32), "UNSUPPORTED"),
                     (dict(dtype=fa.FA_FP16), "UNSUPPORTED")]:
        assert _call(L, "read", **kw) == getattr(fa, "FA_ERR_" + code), kw
    assert _call(L, "read", N=0, k_out=None, v_out=None) == fa.FA_OK
    for kw in (dict(kept=None), dict(counts=None), dict(lens=None), dict(width=-1), dict(kept=FAKE + 1)):
        assert _call(L, "keep", **kw) == fa.FA_ERR_INVALID_ARG, kw
    assert _call(L, "keep", width=0, kept=None) == fa.FA_OK


def test_tree_errors(L):
    n = fa.fa_fwd_tree_workspace_bytes(4, 4, 2, 64)
    for kw, code in [(dict(q=None), "INVALID_ARG"), (dict(o=FAKE + 8), "INVALID_ARG"), (dict(lse=FAKE + 2), "INVALID_ARG"),
                     (dict(q_token_stride=4), "INVALID_ARG"), (dict(o_head_stride=-8), "INVALID_ARG"),
                     (dict(Hq=3), "INVALID_ARG"), (dict(Hq=0), "INVALID_ARG"), (dict(total=-1), "INVALID_ARG"),
                     (dict(max_new=-1), "INVALID_ARG"), (dict(scale=0.0), "INVALID_ARG"),
                     (dict(scale=float("inf")), "INVALID_ARG"), (dict(scale=float("nan")), "INVALID_ARG"),
                     (dict(tree_mask=FAKE, mask_words=0), "INVALID_ARG"),
                     (dict(tree_mask=FAKE, mask_words=1, max_new=65), "INVALID_ARG"),
                     (dict(tree_mask=FAKE + 4, mask_words=1), "INVALID_ARG"),
                     (dict(cu_new=None), "INVALID_ARG"), (dict(lens=FAKE + 2), "INVALID_ARG"),
                     (dict(dtype=fa.FA_FP16), "UNSUPPORTED"), (dict(dtype=fa.FA_FP32), "UNSUPPORTED"),
                     (dict(max_new=2 ** 31 - 1), "UNSUPPORTED"),
                     (dict(workspace=None), "WORKSPACE"), (dict(workspace=FAKE + 16), "WORKSPACE"),
                     (dict(workspace_bytes=n - 1), "WORKSPACE")]:
        assert _call(L, "tree", **kw) == getattr(fa, "FA_ERR_" + code), kw
    assert _call(L, "tree", total=0, q=None, o=None, lse=None, workspace=None) == fa.FA_OK
    assert _call(L, "tree", max_new=0, workspace=None) == fa.FA_OK
    if not torch.cuda.is_available():
        assert _call(L, "tree") == fa.FA_ERR_CUDA


def test_workspace_bytes(L):
    assert fa.fa_fwd_tree_workspace_bytes(1, 8, 3, 64) == 0        # heads that do not divide
    assert fa.fa_fwd_tree_workspace_bytes(1, 8, 2, 96) == 0
    assert fa.fa_fwd_tree_workspace_bytes(-1, 8, 2, 64) == 0
    one = fa.fa_fwd_tree_workspace_bytes(1, 8, 2, 64)
    assert 0 < one <= fa.fa_fwd_tree_workspace_bytes(64, 8, 2, 64)
    assert fa.fa_fwd_tree_workspace_bytes(10 ** 6, 128, 1, 128) < 64 << 20   # does not grow with the call


def test_packed_arguments_have_the_structs_layout():
    c = _cache(k=11, v=12, page_table=13, pages=14)
    for cls, pack, vals in ((fa.CacheAppendArgs, fa._pack_append, [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11]),
                            (fa.CacheReadArgs, fa._pack_read, [1, 2, 3, 4, 5, 6]),
                            (fa.CacheKeepArgs, fa._pack_keep, [1, 2, 3, 4, 5]),
                            (fa.TreeArgs, fa._pack_tree, [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 0.5, 17, 18, 19])):
        got = cls.from_buffer_copy(bytes(c) + pack(*vals))
        assert [getattr(got, n) for n, _ in cls._fields_[1:]] == vals
        assert got.cache.k == 11 and got.cache.pages == 14


def test_python_checks():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.KVCache(k, k, torch.zeros(1, 2, dtype=torch.int32))     # not CUDA tensors


def test_tree_mask_bits():
    cu = torch.tensor([0, 4, 4, 74])
    par = [-1, 0, 0, 1] + [-1] + [i - 1 for i in range(1, 70)]
    m = fa.tree_mask(par, cu)
    assert m.shape == (74, 2) and m.dtype == torch.int64
    bits = m.numpy().astype(np.uint64)
    assert ora.visible(4, bits[:4]).tolist() == [[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 1, 0, 1]]
    assert np.array_equal(ora.visible(70, bits[4:]), np.tril(np.ones((70, 70), dtype=bool)))
    with pytest.raises(ValueError):
        fa.tree_mask([0], torch.tensor([0, 1]))
    with pytest.raises(ValueError):
        fa.tree_mask([-1] * 65, torch.tensor([0, 65]), words=1)


def test_oracle_quantiser_against_torch():
    """Two derivations of the same rows: nearest code by search, and torch's cast of x * 2^-e."""
    g = torch.Generator().manual_seed(0)
    for i in range(40):
        x = (torch.randn(64, generator=g) * 2.0 ** (i - 20)).to(torch.bfloat16)
        codes, s = ora.quantise_row(x.double().numpy(), 240 * 2.0 ** 120)
        want = (x.double() * 2.0 ** (127 - s)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(codes, want)
        amax = float(x.double().abs().max())
        assert amax <= 448 * 2.0 ** (s - 127) < 2 * amax or s == 1
