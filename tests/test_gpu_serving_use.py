"""GPU: the cache operators as a serving program calls them: captured beside copies and forked streams, two graphs at
once, padded batches, layouts and sizes at the ends of their ranges."""

from __future__ import annotations

import pytest
import torch

import exact_attention_111_b200 as fa
from tests.paged import Case, check_attention

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("n", [1, 3, 40])
def test_a_captured_step_with_copies_and_a_forked_stream(n):
    """Append, attention, keep and read between copies, on two streams that part and join inside the graph."""
    c = Case([100, 30, 0], [n, 1, n], 2, 64, 16, BF, True, seed=n, spare=8)
    hk, hv, hq = c.new(2).pin_memory(), c.new(2).pin_memory(), c.new(8).pin_memory()
    k, v, q = (torch.empty_like(x, device="cuda") for x in (hk, hv, hq))
    o, lse = torch.empty_like(q), torch.empty(c.total, 8, device="cuda")
    ws = torch.empty(fa.fa_fwd_tree_workspace_bytes(c.total, 8, 2, 64), dtype=torch.uint8, device="cuda")
    kept = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    counts = torch.ones(3, dtype=torch.int32, device="cuda")
    out = [torch.empty(3, 2, 104, 64, dtype=BF, device="cuda") for _ in range(2)]
    host = torch.empty(o.shape, dtype=BF, pin_memory=True)
    side = torch.cuda.Stream()

    def step():
        now = torch.cuda.current_stream()
        for x, h in ((k, hk), (v, hv), (q, hq)):
            x.copy_(h, non_blocking=True)
        fa.cache_append(c.cache, k, v, c.cu, c.lens)
        side.wait_stream(now)
        with torch.cuda.stream(side):
            fa.cache_read(c.cache, c.lens, 104, k_out=out[0], v_out=out[1])
        fa.attention_forward_tree(q, c.cache, c.cu, c.lens, n, workspace=ws, o=o, lse=lse)
        now.wait_stream(side)
        fa.cache_keep(c.cache, c.lens, kept, counts)
        host.copy_(o, non_blocking=True)

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for h, m in ((hk, 2), (hv, 2), (hq, 8)):
            h.copy_(c.new(m))
        graph.replay()
        fa.fa_check_status()
        check_attention(c, q, o, lse, 1 / 8, label=f"replay {i}")
        torch.cuda.synchronize()
        assert torch.equal(host, o.cpu())
        for x, y in zip(out, fa.cache_read(c.cache, c.lens, 104)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("n", [1, 50])
def test_two_graphs_at_once(n):
    """Two captured calls with their own workspaces, replayed on two streams over one cache."""
    c = Case([900, 64], [n, n], 2, 128, 64, HF, False, seed=4)
    c.put(c.new(2), c.new(2))
    qs = [c.new(8).cuda() for _ in range(2)]
    want = [fa.attention_forward_tree(q, c.cache, c.cu, c.lens, n) for q in qs]
    graphs, got = [], []
    torch.cuda.synchronize()
    for q in qs:
        o, lse = torch.empty_like(q), torch.empty(2 * n, 8, device="cuda")
        ws = torch.empty(fa.fa_fwd_tree_workspace_bytes(2 * n, 8, 2, 128), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fa.attention_forward_tree(q, c.cache, c.cu, c.lens, n, workspace=ws, o=o, lse=lse)
        graphs.append(g)
        got.append((o, lse, ws))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for (o, lse, _), s, g in zip(got, streams, graphs):
            with torch.cuda.stream(s):
                o.fill_(0), lse.fill_(0)
                g.replay()
    torch.cuda.synchronize()
    fa.fa_check_status()
    for (o, lse, _), w in zip(got, want):
        assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
    del graphs


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 7, 60])
def test_tokens_before_the_first_sequence_and_head_major_layouts(n, fp8):
    """cu_new that begins above 0 (tokens in front are padding), q and o with the heads outside."""
    c = Case([50, 300], [n, 1], 2, 64, 16, BF, fp8, seed=n)
    front = 5
    total = c.total + front
    k, v = c.new(2), c.new(2)
    pad = torch.full((front, 2, 64), float("nan"), dtype=BF)
    cu = c.cu + front
    fa.cache_append(c.cache, torch.cat([pad, k]).cuda(), torch.cat([pad, v]).cuda(), cu, c.lens)
    q = torch.full((4, total, 64), float("nan"), dtype=BF, device="cuda")
    q[:, front:] = c.new(4).transpose(0, 1).cuda()
    o = torch.full((4, total, 64), 7.0, dtype=BF, device="cuda")
    lse = torch.full((total, 4), 7.0, device="cuda")
    fa.attention_forward_tree(q.transpose(0, 1), c.cache, cu, c.lens, n, o=o.transpose(0, 1), lse=lse)
    fa.fa_check_status()
    assert torch.all(o[:, :front] == 7) and torch.all(lse[:front] == 7)
    check_attention(c, q[:, front:].transpose(0, 1), o[:, front:].transpose(0, 1), lse[front:], 1 / 8)


def test_outputs_that_overlap_are_refused():
    c = Case([50], [3], 2, 64, 16, BF, False, seed=1)
    c.put(c.new(2), c.new(2))
    q = c.new(4).cuda()
    for o in (torch.empty(1, 4, 64, dtype=BF, device="cuda").expand(3, 4, 64),
              torch.empty(3, 1, 64, dtype=BF, device="cuda").expand(3, 4, 64)):
        with pytest.raises(fa.FAError) as e:
            fa.attention_forward_tree(q, c.cache, c.cu, c.lens, 3, o=o)
        assert e.value.code == fa.FA_ERR_INVALID_ARG
    one = c.new(1)[:, :1].cuda().expand(3, 4, 64)         # queries that are one row: allowed
    o, lse = fa.attention_forward_tree(one, c.cache, c.cu, c.lens, 3)
    fa.fa_check_status()
    check_attention(c, one, o, lse, 1 / 8)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_sequences_of_one_token(fp8):
    """More sequences than the search and the schedule look at in one round (1024), most of them short."""
    B = 1500
    lens = [(7 * b) % 40 for b in range(B)]
    c = Case(lens, [b % 3 != 2 and 1 or 0 for b in range(B)], 1, 64, 16, BF, fp8, seed=1)
    c.put(c.new(1), c.new(1))
    q = c.new(2).cuda()
    o, lse = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, 1)
    fa.fa_check_status()
    check_attention(c, q, o, lse, 1 / 8)
