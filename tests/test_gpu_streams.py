"""GPU: calls on a stream that is not torch's current one, with tensors that the call allocates: they are
the stream's own, so that nothing on another stream is given their memory while the kernels run."""

from __future__ import annotations

import pytest
import torch

import exact_attention_111_b200 as fa
from tests.paged import Case, check_attention
from tests.parity import ensure_built

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _stream_of(t):
    """The stream whose pool of torch's allocator holds t."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("n", [1, 60])
def test_attention_over_the_cache(n, as_handle, monkeypatch):
    c = Case([900, 64], [n, 1], 2, 128, 64, BF, False, seed=4)
    c.put(c.new(2), c.new(2))
    q = c.new(8).cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    scratch = []
    pack = fa._pack_tree
    monkeypatch.setattr(fa, "_pack_tree", lambda *a: scratch.append(a[-3:-1]) or pack(*a))
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)                    # the kernels start after what follows on this stream
    o, lse = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, n, stream=s.cuda_stream if as_handle else s)
    at, size = scratch[0]
    others = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(x.data_ptr() + size <= at or at + size <= x.data_ptr() for x in others)
    assert _stream_of(o) == _stream_of(lse) == s.cuda_stream
    s.synchronize()
    fa.fa_check_status(s)
    check_attention(c, q, o, lse, 1 / 128 ** 0.5)
    k, v = fa.cache_read(c.cache, c.lens, 64, stream=s)
    assert _stream_of(k) == _stream_of(v) == s.cuda_stream
    s.synchronize()
    assert torch.equal(k, fa.cache_read(c.cache, c.lens, 64)[0])
    # the default stream by its handle, from another one
    with torch.cuda.stream(s):
        o2, _ = fa.attention_forward_tree(q, c.cache, c.cu, c.lens, n, stream=0)
    torch.cuda.synchronize()
    assert _stream_of(o2) == 0 and torch.equal(o, o2)


def test_dense_attention():
    ensure_built()
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn(1, 2, 256, 128, generator=g, device="cuda").to(BF) for _ in range(4))
    codes = [x.float().to(torch.float8_e4m3fn) for x in (q, k, v)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()

    def both(f):
        got, want = f(s), f(None)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert _stream_of(x) == s.cuda_stream and _stream_of(y) == torch.cuda.current_stream().cuda_stream
            assert torch.equal(x, y)
        return want

    o, lse = both(lambda st: fa.attention_forward(q, k, v, stream=st))
    both(lambda st: fa.attention_forward_splitkv(q, k, v, num_splits=2, stream=st)[:2])
    parts = both(lambda st: fa.attention_forward_partial(q, k, v, stream=st))
    both(lambda st: fa.lse_merge(parts[:1], parts[1:], stream=st))
    both(lambda st: fa.attention_forward_fp8(*codes, 1.0, 1.0, 1.0, stream=st))
    both(lambda st: fa.attention_backward(q, k, v, o, lse, do, stream=st, deterministic=True))
