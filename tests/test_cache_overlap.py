"""CPU-only: an output whose rows lie on one another is refused."""

from __future__ import annotations

import pytest

import exact_attention_111_b200 as fa
from exact_attention_111_b200 import build as fabuild
from tests.test_cache_args import _call


@pytest.fixture(scope="module")
def L():
    fabuild.build()
    return fa.lib()


def test_outputs_that_overlap(L):
    """d = 64, 4 tokens of 4 heads; without a workspace the next check answers for layouts that will do."""
    for tok, head, ok in [(256, 64, True), (64, 256, True), (264, 64, True), (64, 264, True), (320, 72, True),
                          (0, 64, False), (256, 0, False), (64, 64, False), (128, 64, False), (248, 64, False), (64, 248, False),
                          (56, 1024, False), (1024, 56, False)]:
        got = _call(L, "tree", o_token_stride=tok, o_head_stride=head, workspace=None)
        assert got == (fa.FA_ERR_WORKSPACE if ok else fa.FA_ERR_INVALID_ARG), (tok, head)
    # one token or one head: its stride does not matter
    assert _call(L, "tree", total=1, o_token_stride=0, workspace=None) == fa.FA_ERR_WORKSPACE
    assert _call(L, "tree", cache=dict(Hk=1), Hq=1, o_token_stride=64, o_head_stride=0, workspace=None) == fa.FA_ERR_WORKSPACE
    # queries may be shared
    assert _call(L, "tree", q_token_stride=0, q_head_stride=0, workspace=None) == fa.FA_ERR_WORKSPACE
