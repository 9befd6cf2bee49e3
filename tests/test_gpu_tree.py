"""GPU: attention of new tokens (one, a chain, a drafted tree) over the paged cache against the
fp64 oracle; bounds in tests/paged.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_attention_111_b200 as fa
from tests.paged import Case, check_attention

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _tree(counts, seed):
    """Parents of random trees: the root sees the prefix, later tokens follow an earlier one."""
    rng = np.random.RandomState(seed)
    return [-1 if t == 0 else int(rng.randint(max(0, t - 5), t)) for n in counts for t in range(n)]


def _masks(kind, c, seed):
    if kind == "chain":
        return None
    if kind == "tree":
        return fa.tree_mask(_tree(c.counts_l, seed), c.cu)
    words = (max(c.counts_l) + 63) // 64 + 1            # "random", "holes": any bits, words to spare
    rng = np.random.RandomState(seed)
    m = rng.randint(-2 ** 63, 2 ** 63 - 1, size=(c.total, words), dtype=np.int64)
    if kind == "holes":
        m[rng.rand(c.total) < 0.5] = 0                   # rows that see no new token
    return torch.from_numpy(m).cuda()


CASES = [
    # lens, counts, Hq, Hk, d, page, dtype, fp8, mask
    ([0], [1], 1, 1, 64, 16, BF, False, "chain"),
    ([1], [1], 4, 1, 128, 16, HF, False, "chain"),
    ([15, 16, 17, 0, 127], [1] * 5, 8, 8, 64, 16, HF, False, "chain"),
    ([300, 5, 1030, 128], [1] * 4, 32, 8, 128, 64, BF, False, "chain"),
    ([700, 129], [1, 1], 48, 3, 128, 32, BF, False, "chain"),
    ([2500], [1], 8, 1, 64, 128, HF, False, "chain"),
    ([90, 0, 33], [5, 7, 2], 6, 2, 64, 16, BF, False, "chain"),
    ([64, 200], [19, 3], 14, 2, 128, 64, HF, False, "tree"),
    ([120, 0, 3], [40, 0, 65], 8, 2, 128, 32, BF, False, "tree"),
    ([0, 50], [30, 9], 4, 4, 64, 16, HF, False, "holes"),
    ([200], [70], 3, 1, 128, 128, BF, False, "random"),
    ([0, 70], [150, 33], 10, 2, 64, 64, HF, False, "chain"),
    ([0], [1], 2, 1, 128, 16, HF, True, "chain"),
    ([15, 400, 16], [1] * 3, 16, 2, 128, 16, BF, True, "chain"),
    ([33, 900, 1], [1] * 3, 8, 8, 64, 32, HF, True, "chain"),
    ([500, 20], [1, 1], 5, 1, 64, 128, BF, True, "chain"),
    ([77, 130], [24, 11], 12, 4, 128, 64, HF, True, "tree"),
    ([0, 256], [12, 66], 16, 2, 64, 16, BF, True, "tree"),
    ([0, 9], [20, 5], 21, 3, 128, 16, BF, True, "holes"),
    ([40], [100], 7, 1, 128, 128, HF, True, "chain"),
    ([5] * 40, [1, 2] * 20, 4, 2, 64, 16, BF, False, "tree"),
    # many rows of a key head: several row tiles, units cut between CTAs
    ([1000, 20, 0], [64, 129, 1], 16, 2, 128, 16, BF, False, "chain"),
    ([700], [130], 12, 2, 64, 32, HF, False, "random"),
    ([0, 513], [33, 64], 24, 3, 128, 128, HF, False, "tree"),
    ([127, 128], [90, 91], 7, 1, 64, 128, BF, False, "holes"),
    ([600, 3], [140, 70], 8, 2, 128, 64, HF, True, "tree"),
    ([30, 400], [150, 64], 4, 1, 64, 16, BF, True, "chain"),
]


@pytest.mark.parametrize("lens,counts,Hq,Hk,d,page,dtype,fp8,mask", CASES)
def test_matches_oracle(lens, counts, Hq, Hk, d, page, dtype, fp8, mask):
    c = Case(lens, counts, Hk, d, page, dtype, fp8, seed=sum(lens) + Hq + d)
    c.put(c.new(Hk), c.new(Hk))
    pad = 3
    q = torch.cat([c.new(Hq + 2), torch.full((pad, Hq + 2, d), float("nan"), dtype=dtype)]).cuda()[:, 1:1 + Hq]
    bits = _masks(mask, c, seed=Hq)
    if bits is not None:
        bits = torch.cat([bits, torch.full((pad, bits.shape[1]), -1, dtype=torch.int64, device="cuda")])
    big = torch.full((c.total + pad, Hq + 1, d), 7.0, dtype=dtype, device="cuda")
    o, lse = big[:, :Hq], torch.full((c.total + pad, Hq), 7.0, device="cuda")
    ws = torch.full((fa.fa_fwd_tree_workspace_bytes(c.total + pad, Hq, Hk, d) // 4,), float("nan"), device="cuda")
    fa.attention_forward_tree(q, c.cache, c.cu, c.lens, max(counts), tree_mask=bits, o=o, lse=lse, workspace=ws)
    fa.fa_check_status()
    check_attention(c, q[:c.total], o[:c.total], lse[:c.total], 1 / d ** 0.5, None if bits is None else bits[:c.total],
                    f"{mask} fp8={fp8}")
    assert torch.all(big[c.total:] == 7) and torch.all(lse[c.total:] == 7) and torch.all(big[:, Hq] == 7)
    o2, lse2 = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, max(counts), tree_mask=bits)
    fa.fa_check_status()
    assert torch.equal(o2[:c.total], o[:c.total]) and torch.equal(lse2[:c.total], lse[:c.total])   # repeatable


@pytest.mark.parametrize("G,n", [(1, 20), (4, 20), (8, 40)])
@pytest.mark.parametrize("dtype,fp8", [(BF, False), (HF, False), (BF, True), (HF, True)])
def test_values_a_row_does_not_see_do_not_reach_it(G, n, dtype, fp8):
    """New tokens' K and V that are not finite: rows that see them get what the definition gives,
    the others nothing of it."""
    c = Case([37], [n], 2, 64, 16, dtype, fp8, seed=G)
    k, v = c.new(2), c.new(2)
    for t, x in ((3, float("nan")), (7, float("inf")), (11, -float("inf"))):
        v[t, :, t::5] = x
    k[15] = float("nan")
    c.put(k, v)
    q = c.new(2 * G).cuda()
    par = [-1] + [0] * (n - 1)                           # a star: siblings do not see one another
    par[n - 1] = 7
    bits = fa.tree_mask(par, c.cu)
    o, lse = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, n, tree_mask=bits)
    fa.fa_check_status()
    check_attention(c, q, o, lse, 1 / 8, bits, nan_ok=True)


@pytest.mark.parametrize("n", [2, 40])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_nan_codes_of_the_prefix(dtype, n):
    """A NaN in the prefix reaches every row's result (V: its column) and nothing hides it."""
    c = Case([200], [n], 2, 64, 16, dtype, True, seed=5)
    c.put(c.new(2), c.new(2))
    p, r = c.table_np[0, 3], 5
    c.gpu["v"][p, 0, r, 17] = 127
    c.gpu["k"][p, 1, r, 9] = 255
    q = c.new(4).cuda()
    o, lse = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, n)
    fa.fa_check_status()
    check_attention(c, q, o, lse, 1 / 8, nan_ok=True)
    assert torch.isnan(o[:, :2, 17]).all() and torch.isnan(o[:, 2:]).all()


@pytest.mark.parametrize("mask", ["chain", "random"])
@pytest.mark.parametrize("n", [3, 40, 300])
@pytest.mark.parametrize("dtype,fp8", [(BF, False), (HF, False), (BF, True), (HF, True)])
def test_values_of_the_prefix_beside_new_tokens(dtype, fp8, n, mask):
    """Prefix keys in the same block of keys as the first new tokens: NaN and infinities there reach
    every row, also where the block's masked products are made safe."""
    c = Case([200], [n], 2, 64, 16, dtype, fp8, seed=n)
    c.put(c.new(2), c.new(2))
    for pos, col, x in ((199, 5, float("nan")), (193, 9, float("inf")), (140, 40, -float("inf"))):
        p, r = c.table_np[0, pos // 16], pos % 16
        c.gpu["v"][p, 1, r, col] = 127 if fp8 else x
    q = c.new(4).cuda()
    bits = _masks(mask, c, seed=1)
    o, lse = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, n, tree_mask=bits)
    fa.fa_check_status()
    check_attention(c, q, o, lse, 1 / 8, bits, nan_ok=True)
    assert not torch.isfinite(o[:, 2:, [5, 9, 40]]).any()


@pytest.mark.parametrize("d,fp8,T,G", [(64, True, 250, 12), (128, True, 250, 12), (64, False, 250, 12), (64, True, 40, 5),
                                       (64, True, 1, 4), (128, True, 1, 8)])
def test_many_short_units_many_times(d, fp8, T, G):
    """Units of a few tiles each, so that every role of the kernel runs ahead of the others and across
    units; the results are the same bits every time, and right."""
    counts = [max(1, T - 10 * b) for b in range(7)]
    c = Case([79, 80, 161, 120, 125, 113, 129], counts, 5, d, 128, BF, fp8, seed=T + d)
    c.put(c.new(5), c.new(5))
    q = c.new(5 * G).cuda()
    o, lse = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, T)
    K, V = (torch.from_numpy(x).cuda() for x in c.values())
    for b in range(c.B):                                 # fp64 on the GPU: the same definition, no bound per row
        n, a, e = c.lens_l[b] + counts[b], c.cu_l[b], c.cu_l[b + 1]
        pos = torch.arange(n)
        pg, r = torch.from_numpy(c.table_np[b][pos // 128]).long().cuda(), (pos % 128).cuda()
        k, v = (x[pg, :, r].transpose(0, 1) for x in (K, V))
        x = torch.einsum("tgd,gnd->gtn", q[a:e].double().view(-1, 5, G, d).transpose(1, 2).reshape(-1, 5, d),
                         k).div(d ** 0.5).view(5, e - a, G, n)
        seen = torch.arange(n, device="cuda")[None, :] <= c.lens_l[b] + torch.arange(e - a, device="cuda")[:, None]
        p = torch.softmax(x.masked_fill(~seen[None, :, None], float("-inf")), -1)
        want = torch.einsum("gtkn,gnd->tgkd", p, v).reshape(e - a, 5 * G, d)
        # P and O rounded to bf16: 2 * 2^-8 of sum p |v| <= max |v| over the visible keys
        bound = 2.1 * 2.0 ** -8 * float(v.abs().max())
        assert float((o[a:e].double() - want).abs().max()) <= bound
    for _ in range(30):
        o2, lse2 = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, T)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    fa.fa_check_status()


def test_rows_behind_four_gigabytes():
    """A cache whose K and V are over 4 GB each: positions in its last pages."""
    pages, Hk, page, d = 40000, 8, 64, 128
    k = torch.empty(pages, Hk, page, d, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    assert k.numel() * 2 > 2 ** 32
    g = torch.Generator().manual_seed(2)
    small = Case([150], [3], Hk, d, page, BF, False, seed=3)          # the same sequence in a small cache
    big_table = torch.tensor([[pages - 1, pages - 5, pages - 2, 0]], dtype=torch.int32, device="cuda")
    for e in range(3):
        k[big_table[0, e]] = small.gpu["k"][small.table_np[0, e]]
        v[big_table[0, e]] = small.gpu["v"][small.table_np[0, e]]
    big = fa.KVCache(k, v, big_table)
    kn, vn = (torch.randn(3, Hk, d, generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn(3, 16, d, generator=g).to(BF).cuda()
    one = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")[None, 1:].contiguous()
    two = torch.tensor([2], dtype=torch.int32, device="cuda")
    for cache in (small.cache, big):
        fa.cache_append(cache, kn, vn, small.cu, small.lens)
    a = fa.attention_forward_tree(q, small.cache, small.cu, small.lens, 3)
    b = fa.attention_forward_tree(q, big, small.cu, small.lens, 3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_attention(small, q, *a, 1 / d ** 0.5)
    one[0, 1] = 2
    for cache in (small.cache, big):
        fa.cache_keep(cache, small.lens, one, two)
    x, y = (fa.cache_read(cache, small.lens + 2, 152) for cache in (small.cache, big))
    fa.fa_check_status()
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("fp8", [False, True])
def test_long_peaked_rows(fp8, n):
    """Scores in the tens: the running max changes all the way."""
    c = Case([2000], [n], 1, 128, 64, BF, fp8, seed=9, k_gain=4.0 if not fp8 else 1.0)
    c.put(c.new(1), c.new(1))
    q = (c.new(4) * 4).cuda()
    o, lse = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, n)
    fa.fa_check_status()
    check_attention(c, q, o, lse, 1 / 128 ** 0.5)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n", [1, 48])
def test_scales_that_differ_widely_along_the_keys(dtype, n):
    """K and V rows whose magnitudes rise by steps of up to 2^12 along the keys and fall again, and rows
    of zeros: every rescale of the E4M3 path."""
    c = Case([700], [n], 1, 64, 16, dtype, True, seed=6)
    c.put(c.new(1), c.new(1))
    for p in range(700):
        i, r = c.table_np[0, p // 16], p % 16
        up = (0, 3, 9, 12, 24, 13, -6)[p // 100]
        c.gpu["v_scale"][i, :, r] = 112 + up - (5 if p % 3 else 0)
        c.gpu["k_scale"][i, :, r] = 118 - (6 if p % 5 else 0) + (2 if p > 500 else 0)
        if p % 50 == 0:
            c.gpu["v"][i, :, r] = 0
            c.gpu["v_scale"][i, :, r] = 1
    q = c.new(2).cuda()
    o, lse = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, n)
    fa.fa_check_status()
    check_attention(c, q, o, lse, 1 / 8)


def test_bf16_queries_of_any_size_over_codes():
    """Rows of Q far outside fp16's range (their products are made in fp16)."""
    for n in (2, 40):
        c = Case([300], [n], 1, 64, 16, BF, True, seed=8)
        c.gpu["k_scale"].fill_(60)
        c.put((c.new(1).float() * 2.0 ** -60).to(BF), c.new(1))
        q = (c.new(1).float() * 2.0 ** 60).to(BF)
        q[1] = 0
        q = q.cuda()
        o, lse = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, n)
        fa.fa_check_status()
        check_attention(c, q, o, lse, 1 / 8)


def test_lengths_on_the_device_are_what_a_replayed_graph_reads():
    """One captured step, replayed with other lengths and tokens."""
    c = Case([100, 30, 0], [1, 1, 1], 2, 64, 16, BF, True, seed=21, spare=40)
    free = sorted(set(range(c.pages)) - set(c.table_np.ravel().tolist()))     # pages to grow into
    for i, (b, e) in enumerate(np.argwhere(c.table_np < 0)):
        c.table_np[b, e] = free[i]
    q, k, v = (x.cuda() for x in (c.new(8), c.new(2), c.new(2)))
    c.table.copy_(torch.from_numpy(c.table_np))
    lens = c.lens.clone()
    o, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
    ws = torch.empty(fa.fa_fwd_tree_workspace_bytes(3, 8, 2, 64), dtype=torch.uint8, device="cuda")

    def step():
        fa.cache_append(c.cache, k, v, c.cu, lens)
        fa.attention_forward_tree(q, c.cache, c.cu, lens, 1, workspace=ws, o=o, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(5):
        c.lens_l = [c.lens_l[0] + 1, c.lens_l[1] + 1, c.lens_l[2] + 1]
        lens.add_(1)
        q.copy_(c.new(8)), k.copy_(c.new(2)), v.copy_(c.new(2))
        graph.replay()
        fa.fa_check_status()
        check_attention(c, q, o, lse, 1 / 8, label=f"replay {i}")


def test_two_streams_with_their_own_workspaces():
    c = Case([900, 64], [1, 1], 2, 128, 64, BF, False, seed=4)
    c.put(c.new(2), c.new(2))
    q = c.new(8).cuda()
    want = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, 1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append([fa.attention_forward_tree(q, c.cache, c.cu, c.lens, 1) for _ in range(20)])
    torch.cuda.synchronize()
    for run in got:
        for o, lse in run:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_a_drafted_step_end_to_end():
    """Draft a tree, attend, keep a path, attend with the next token: the same as a sequence that
    was written token by token; and what is read back gives the dense forward's result."""
    c = Case([50, 33], [9, 6], 2, 128, 16, BF, True, seed=12, spare=8)
    k, v, q = c.new(2), c.new(2), c.new(8).cuda()
    c.put(k, v)
    par = [-1, 0, 0, 1, 1, 2, 3, 4, 6] + [-1, 0, 1, 0, 3, 3]
    bits = fa.tree_mask(par, c.cu)
    o, lse = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, 9, tree_mask=bits)
    check_attention(c, q, o, lse, 1 / 128 ** 0.5, bits)
    path = [[0, 1, 3, 6, 8], [0, 3, 5]]
    kept = torch.tensor([p + [0] * (5 - len(p)) for p in path], dtype=torch.int32).cuda()
    counts = torch.tensor([5, 3], dtype=torch.int32).cuda()
    fa.cache_keep(c.cache, c.lens, kept, counts)
    # the same path written as a chain into another cache
    r = Case([50, 33], [5, 3], 2, 128, 16, BF, True, seed=12, spare=20)
    idx = torch.tensor(path[0] + [9 + t for t in path[1]])
    fa.cache_append(r.cache, k[idx].cuda(), v[idx].cuda(), r.cu, r.lens)
    o2, lse2 = fa.attention_forward_tree(q[idx.cuda()].contiguous(), r.cache, r.cu, r.lens, 5)
    fa.fa_check_status()
    check_attention(r, q[idx.cuda()], o2, lse2, 1 / 128 ** 0.5)
    ends = c.lens + counts
    a, b = fa.cache_read(c.cache, ends, 55), fa.cache_read(r.cache, r.lens + counts, 55)
    for s, n0, n in ((0, 50, 5), (1, 33, 3)):
        for x, y in zip(a, b):
            assert torch.equal(x[s, :, n0:n0 + n], y[s, :, n0:n0 + n])
    # dense attention of the last accepted token over what was read back
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    last = torch.stack([q[8], q[9 + 5]])
    o3, lse3 = fa.attention_forward_tree(last, c.cache, cu, ends - 1, 1)
    for s, n in ((0, 55), (1, 36)):
        kk = a[0][s:s + 1, :, :n].repeat_interleave(4, 1).contiguous()
        vv = a[1][s:s + 1, :, :n].repeat_interleave(4, 1).contiguous()
        od, ld = fa.attention_forward_partial(last[s].view(1, 8, 1, 128).contiguous(), kk, vv)
        # the same values through two kernels: P rounded to bf16 in each (2^-8 of sum p |v| <=
        # max |v|), the result once more in one
        bound = 2 * 2.0 ** -8 * float(vv.abs().max()) + 2.0 ** -8 * float(od.abs().max())
        assert (o3[s].float() - od.view(8, 128)).abs().max() <= bound
        assert (lse3[s] - ld.view(8)).abs().max() <= 1e-4
    fa.fa_check_status()


def test_lengths_that_cannot_be_are_reported():
    c = Case([20, 20], [2, 2], 2, 64, 16, BF, False, seed=3)
    c.put(c.new(2), c.new(2))
    q = c.new(4).cuda()

    def refused(cu=c.cu, lens=c.lens, max_new=2):
        fa.attention_forward_tree(q, c.cache, cu, lens, max_new)
        with pytest.raises(fa.FAError) as e:
            fa.fa_check_status()
        assert e.value.code == fa.FA_ERR_RANGE

    refused(lens=torch.tensor([20, -1], dtype=torch.int32).cuda())
    refused(lens=torch.tensor([20, 2 ** 30], dtype=torch.int32).cuda())
    refused(lens=torch.tensor([2 ** 31 - 1, 1], dtype=torch.int32).cuda())
    refused(cu=torch.tensor([0, 2, 5], dtype=torch.int32).cuda())
    refused(cu=torch.tensor([-1, 1, 2], dtype=torch.int32).cuda())
    refused(cu=torch.tensor([0, 3, 2], dtype=torch.int32).cuda(), max_new=4)
    refused(max_new=1)
    table = c.table.clone()
    for bad in (-1, c.pages, 2 ** 31 - 1):
        c.table[1, 0] = bad
        refused()
        c.table.copy_(table)
    o, lse = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, 2)
    fa.fa_check_status()
    check_attention(c, q, o, lse, 1 / 8)


@pytest.mark.parametrize("d,dtype,fp8", [(64, HF, False), (128, BF, False), (64, BF, True), (128, HF, True)])
def test_units_that_end_anywhere_in_a_warp(d, dtype, fp8):
    """Many-row units whose last warp has from one to all 32 of its rows, in whole units and in units cut
    between CTAs, with values that are not finite: what the whole warp loads and what its rows do apart."""
    for T in (33, 34, 47, 63, 64, 65, 95, 127, 129, 130, 159, 193, 255):
        c = Case([3, 700], [T, T - 1], 1, d, 16, dtype, fp8, seed=T + d)
        k, v = c.new(1), c.new(1)
        for t, x in ((1, float("nan")), (T // 2, float("inf")), (T + 5, -float("inf"))):
            v[t, :, t % 7::9] = x
        c.put(k, v)
        q = c.new(1).cuda()
        bits = _masks("random", c, seed=T)
        o, lse = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, T, tree_mask=bits)
        fa.fa_check_status()
        check_attention(c, q, o, lse, 1 / d ** 0.5, bits, f"T={T}", nan_ok=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_max_new_of_zero(fp8):
    """It says that no sequence has new tokens: true for a batch that is all padding, whose results stay as they
    were, and reported where a sequence has some."""
    c = Case([20, 300], [2, 2], 2, 64, 16, BF, fp8, seed=3)
    c.put(c.new(2), c.new(2))
    q = c.new(4).cuda()
    o, lse = torch.full_like(q, 7), torch.full((4, 4), 7.0, device="cuda")
    empty = torch.full_like(c.cu, 4)
    fa.attention_forward_tree(q, c.cache, empty, c.lens, 0, o=o, lse=lse)
    fa.fa_check_status()
    assert torch.all(o == 7) and torch.all(lse == 7)
    for mask in (None, torch.zeros(4, 1, dtype=torch.int64, device="cuda")):
        fa.attention_forward_tree(q, c.cache, c.cu, c.lens, 0, tree_mask=mask, o=o, lse=lse)
        with pytest.raises(fa.FAError) as e:
            fa.fa_check_status()
        assert e.value.code == fa.FA_ERR_RANGE
    fa.attention_forward_tree(q, c.cache, c.cu, c.lens, 2, o=o, lse=lse)
    fa.fa_check_status()
    check_attention(c, q, o, lse, 1 / 8)
