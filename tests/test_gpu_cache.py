"""GPU: the paged cache -- rows quantised as they are written, read back, and kept -- against the
fp64 oracle.  Quantising has one right answer for every code, so the comparison is for equality."""

from __future__ import annotations

import copy

import numpy as np
import pytest
import torch

import exact_attention_111_b200 as fa
import oracle.paged as ora
from tests.paged import TOP, Case

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _bits(t):
    return t.cpu().contiguous().view(torch.uint8).numpy()


CASES = [
    # lens, counts, Hk, d, page, dtype, fp8
    ([0], [1], 1, 64, 16, BF, True),
    ([5, 0, 31], [1, 1, 1], 8, 128, 16, BF, True),
    ([100, 15, 16, 17], [3, 0, 33, 1], 3, 64, 32, HF, True),
    ([7, 250], [140, 5], 5, 128, 128, HF, True),
    ([0, 9, 63], [64, 1, 2], 2, 128, 64, BF, False),
    ([40, 3], [1, 29], 7, 64, 16, HF, False),
    ([3] * 70, [1, 0] * 35, 1, 128, 16, BF, True),
]


def _expect_append(c, k_new, v_new):
    want = {n: x.clone() for n, x in c.t.items()}
    for n, x in (("k", k_new), ("v", v_new)):
        for b in range(c.B):
            for i in range(c.counts_l[b]):
                p, r = ora.slot(c.table_np, b, c.lens_l[b] + i, c.page)
                for h in range(c.Hk):
                    row = x[c.cu_l[b] + i, h]
                    if c.fp8:
                        codes, s = ora.quantise_row(row.double().numpy(), TOP[c.dtype])
                        want[n][p, h, r] = torch.from_numpy(codes)
                        want[n + "_scale"][p, h, r] = s
                    else:
                        want[n][p, h, r] = row
    return want


@pytest.mark.parametrize("lens,counts,Hk,d,page,dtype,fp8", CASES)
def test_append_writes_the_rows_and_nothing_else(lens, counts, Hk, d, page, dtype, fp8):
    c = Case(lens, counts, Hk, d, page, dtype, fp8, seed=len(lens) + d + page)
    fused = c.new(3 * Hk + 1, pad=5)                     # K and V inside one projection, padded tokens behind
    k_new, v_new = fused[:, 1:1 + Hk], fused[:, 1 + Hk:1 + 2 * Hk]
    gk = fused.cuda()
    fa.cache_append(c.cache, gk[:, 1:1 + Hk], gk[:, 1 + Hk:1 + 2 * Hk], c.cu, c.lens)
    fa.fa_check_status()
    want = _expect_append(c, k_new, v_new)
    for n in want:
        assert np.array_equal(_bits(c.gpu[n]), _bits(want[n])), n
    assert c.lens.tolist() == c.lens_l


@pytest.mark.parametrize("dtype", [BF, HF])
def test_quantised_extremes(dtype):
    """Zeros, subnormals, the largest values, powers of two about the scale's steps, ties, NaN and
    infinities."""
    d = 64
    big = torch.finfo(dtype).max
    tiny = torch.finfo(dtype).smallest_normal
    rows = torch.zeros(12, 1, d)
    rows[1, 0, 3] = tiny / 2 ** 6
    rows[2, 0] = torch.linspace(-1, 1, d)
    rows[3, 0, :4] = torch.tensor([448.0, 447.0, -448.0, 2.0 ** -9])
    rows[4, 0, :4] = torch.tensor([449.0, 450.0, -451.0, 1.0])          # rounds to 448 and 450 in bf16 / fp16
    rows[5, 0, :5] = torch.tensor([256.0, 17.0, 19.0, 21.0, -23.0])      # ties between E4M3 neighbours
    rows[6, 0, :3] = torch.tensor([big, -big, big / 2])
    rows[7, 0, :4] = torch.tensor([float("nan"), 1.0, -2.0, 3.0])
    rows[8, 0, :4] = torch.tensor([float("inf"), -float("inf"), 0.5, 448.0])
    rows[9, 0] = float("nan")
    rows[10, 0, :2] = torch.tensor([-0.0, 2.0 ** -14])
    rows[11, 0] = torch.arange(d) * 1.75
    x = rows.to(dtype)
    c = Case([0], [12], 1, d, 16, dtype, True, seed=1)
    fa.cache_append(c.cache, x.cuda(), x.flip(0).contiguous().cuda(), c.cu, c.lens)
    fa.fa_check_status()
    want = _expect_append(c, x, x.flip(0))
    for n in want:
        assert np.array_equal(_bits(c.gpu[n]), _bits(want[n])), n
    # what is stored is finite in the source's type where the source was
    k, _ = fa.cache_read(c.cache, c.lens + 12, 12, dtype=dtype)
    assert torch.equal(torch.isfinite(k.cpu()[0, 0]), torch.isfinite(x[:, 0]))


@pytest.mark.parametrize("lens,counts,Hk,d,page,dtype,fp8", CASES)
def test_read_gives_the_values_and_zeros_past_the_end(lens, counts, Hk, d, page, dtype, fp8):
    c = Case(lens, counts, Hk, d, page, dtype, fp8, seed=7 * len(lens) + d)
    N = max(lens) + 3                                   # odd, past every end, not a multiple of anything
    K, V = c.values()
    for out in ([BF, HF] if fp8 else [dtype]):
        k, v = fa.cache_read(c.cache, c.lens, N, dtype=out)
        fa.fa_check_status()
        for got, x in ((k, K), (v, V)):
            want = np.zeros((c.B, Hk, N, d))
            for b in range(c.B):
                want[b, :, :lens[b]] = ora.gather(x, c.table_np, b, lens[b], page)
            assert torch.equal(got.cpu(), torch.from_numpy(want).to(out))
    short = max(lens) // 2
    if short:
        k2, _ = fa.cache_read(c.cache, c.lens, short, dtype=dtype)
        k1, _ = fa.cache_read(c.cache, c.lens, N, dtype=dtype)
        assert torch.equal(k2, k1[:, :, :short])


@pytest.mark.parametrize("d,page,dtype,fp8", [(64, 16, HF, True), (128, 64, BF, True), (128, 16, BF, False),
                                              (64, 128, HF, False)])
def test_keep_moves_the_accepted_rows(d, page, dtype, fp8):
    lens, counts = [0, 13, 40, 16, 7], [1, 40, 70, 3, 5]
    c = Case(lens, counts, 3, d, page, dtype, fp8, seed=d + page)
    c.put(c.new(3), c.new(3))
    kept = [[0], [0, 1, 5, 6, 20, 39], list(range(0, 70, 2)) + [69], [], [4]]
    width = max(map(len, kept)) + 2
    before = {n: x.cpu().clone() for n, x in c.gpu.items()}
    kt = torch.full((5, width), -7, dtype=torch.int32)   # entries past the count are not looked at
    for b, row in enumerate(kept):
        kt[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
    fa.cache_keep(c.cache, c.lens, kt.cuda(), torch.tensor(list(map(len, kept)), dtype=torch.int32).cuda())
    fa.fa_check_status()
    want = {n: x.clone() for n, x in before.items()}
    for b, row in enumerate(kept):
        for i, t in enumerate(row):
            (p0, r0), (p1, r1) = (ora.slot(c.table_np, b, lens[b] + j, page) for j in (t, i))
            for n in want:
                want[n][p1, :, r1] = before[n][p0, :, r0]
    for n in want:
        assert np.array_equal(_bits(c.gpu[n]), _bits(want[n])), n


def _range_error():
    with pytest.raises(fa.FAError) as e:
        fa.fa_check_status()
    assert e.value.code == fa.FA_ERR_RANGE
    fa.fa_check_status()                                 # reported once


def test_bad_pages_and_lists_are_reported_and_touch_nothing():
    c = Case([20, 20], [4, 4], 2, 64, 16, BF, True, seed=3)
    before = {n: x.clone() for n, x in c.gpu.items()}
    k, v = c.new(2).cuda(), c.new(2).cuda()
    good = c.table.clone()
    for bad in (-1, c.pages, 2 ** 31 - 1):
        c.table.copy_(good)
        c.table[:, 1] = bad                              # positions 16 .. 31: where the new rows go
        fa.cache_append(c.cache, k, v, c.cu, c.lens)
        _range_error()
        kk, _ = fa.cache_read(c.cache, c.lens, 20)
        _range_error()
        assert torch.all(kk[:, :, 16:] == 0)
    c.table.copy_(good)
    past = torch.full_like(c.lens, 16 * c.table.shape[1])
    fa.cache_append(c.cache, k, v, c.cu, past)
    _range_error()
    fa.cache_append(c.cache, k, v, c.cu, torch.full_like(c.lens, -1))
    _range_error()
    two = torch.full((2,), 2, dtype=torch.int32, device="cuda")
    for rows in ([[1, 1], [1, 1]], [[2, 1], [2, 1]], [[-1, 0], [-1, 0]]):
        fa.cache_keep(c.cache, c.lens, torch.tensor(rows, dtype=torch.int32).cuda(), two)
        _range_error()
    fa.cache_keep(c.cache, c.lens, torch.zeros(2, 1, dtype=torch.int32).cuda(), two)      # count > width
    _range_error()
    fa.cache_keep(c.cache, past, torch.tensor([[0, 1]] * 2, dtype=torch.int32).cuda(), two)
    _range_error()
    for n in before:
        assert torch.equal(before[n], c.gpu[n]), n


@pytest.mark.parametrize("fp8", [False, True])
def test_the_tensors_of_a_cache_are_fixed(fp8):
    """The calls use the addresses that the KVCache took, so no other tensor can be put in one's place, and a
    copy has its own."""
    c = Case([20, 3], [2, 1], 2, 64, 16, BF, fp8, seed=3)
    for name in ("k", "v", "k_scale", "v_scale", "page_table", "pages", "B", "args"):
        with pytest.raises(AttributeError):
            setattr(c.cache, name, None)
        with pytest.raises(AttributeError):
            delattr(c.cache, name)
    c.cache.layer = 3                                    # the caller's own
    wide = torch.cat([c.table, c.table[:, :1]], 1).contiguous()
    bigger = fa.KVCache(c.cache.k, c.cache.v, wide, c.cache.k_scale, c.cache.v_scale)
    assert bigger.max_pages == c.cache.max_pages + 1
    other = copy.deepcopy(c.cache)
    assert other.k.data_ptr() != c.cache.k.data_ptr() and other.args != c.cache.args
    before = {n: _bits(x) for n, x in c.gpu.items()}
    k, v = c.new(2).cuda(), c.new(2).cuda()
    fa.cache_append(other, k, v, c.cu, c.lens)           # the copy's rows, not the first cache's
    for n in before:
        assert np.array_equal(before[n], _bits(c.gpu[n])), n
    fa.cache_append(c.cache, k, v, c.cu, c.lens)
    fa.fa_check_status()
    for n in before:
        assert np.array_equal(_bits(getattr(other, n)), _bits(c.gpu[n])), n


@pytest.mark.parametrize("fp8", [False, True])
def test_append_reports_bounds_that_cannot_be(fp8):
    """New-token bounds outside 0 .. total, and lists that decrease: reported, and no row goes to a slot that is
    not its own."""
    c = Case([20, 20, 7], [2, 2, 0], 2, 64, 16, BF, fp8, seed=3)
    k, v = c.new(2), c.new(2)
    gk, gv = k.cuda(), v.cuda()
    want = _expect_append(c, k, v)
    before = {n: _bits(x) for n, x in c.gpu.items()}
    wrong = [[-1, 2, 4, 4], [-1, 1, 3, 4], [0, 2, 5, 5], [0, 3, 2, 4], [2, 0, 4, 4], [0, 2, 4, 3], [0, 2, 4, 2 ** 31 - 1],
             [-2 ** 31, 2, 4, 4]]
    for cu in wrong:
        for n, x in c.gpu.items():
            x.copy_(torch.from_numpy(before[n]).view(x.dtype).view(x.shape))
        fa.cache_append(c.cache, gk, gv, torch.tensor(cu, dtype=torch.int32).cuda(), c.lens)
        _range_error()
        for b in range(3):
            for pos in range(c.lens_l[b]):               # what a sequence holds stays
                p, r = ora.slot(c.table_np, b, pos, c.page)
                for n, x in c.gpu.items():
                    was = torch.from_numpy(before[n]).view(x.dtype).view(x.shape)
                    assert np.array_equal(_bits(x[p, :, r]), _bits(was[p, :, r])), (cu, b, pos, n)
    for n, x in c.gpu.items():
        x.copy_(torch.from_numpy(before[n]).view(x.dtype).view(x.shape))
    fa.cache_append(c.cache, gk, gv, c.cu, c.lens)
    fa.fa_check_status()
    for n in want:
        assert np.array_equal(_bits(c.gpu[n]), _bits(want[n])), n
    # a padded batch: tokens in front of the first sequence and behind the last are ignored
    some = torch.tensor([1, 2, 3, 3], dtype=torch.int32).cuda()
    fa.cache_append(c.cache, gk, gv, some, c.lens)
    fa.fa_check_status()


@pytest.mark.parametrize("out", [BF, HF])
def test_every_code_and_scale_is_read_as_what_it_stands_for(out):
    """All 256 codes under all scale codes from 0 (2^-127) to 254."""
    d, page = 64, 128
    codes = torch.arange(256, dtype=torch.uint8).view(4, d).repeat(255, 1).cuda()          # row 4 s + i: scale s
    scales = torch.arange(255, dtype=torch.uint8).repeat_interleave(4).cuda()
    N = codes.shape[0]
    pages = -(-N // page)
    k = torch.zeros(pages, 1, page, d, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(pages, 1, page, dtype=torch.uint8, device="cuda")
    k.view(-1, d)[:N], ks.view(-1)[:N] = codes, scales
    cache = fa.KVCache(k, k.clone(), torch.arange(pages, dtype=torch.int32, device="cuda")[None], ks, ks.clone())
    got = fa.cache_read(cache, torch.tensor([N], dtype=torch.int32, device="cuda"), N, dtype=out)
    fa.fa_check_status()
    want = ora.e4m3_values(codes.cpu().numpy()) * np.exp2(scales.cpu().numpy().astype(np.float64) - 127)[:, None]
    want = torch.from_numpy(want).to(out)
    for x in got:
        x = x.cpu()[0, 0]
        assert torch.equal(torch.isnan(x), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(x, nan=0.0), torch.nan_to_num(want, nan=0.0))
