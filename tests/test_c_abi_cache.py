"""The C entry points of the paged cache as a C program and as the Python calls of the same names reach them."""

from __future__ import annotations

import os
import shutil
import subprocess
import tempfile

import pytest
import torch

import exact_attention_111_b200 as fa
from exact_attention_111_b200 import build as fabuild
from tests.test_cache_args import FAKE, _cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("gcc") is None, reason="no C compiler")
def test_c_program():
    lib = fabuild.build()
    libdir = os.path.dirname(lib)
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "cache_check")
        subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                        os.path.join(ROOT, "tests", "c_abi", "cache_check.c"), "-o", exe, "-L", libdir, "-l:libfa.so",
                        f"-Wl,-rpath,{libdir}"], check=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stdout + r.stderr
        assert "c abi ok" in r.stdout


def test_python_calls_report_refusals():
    fabuild.build()
    c, st = bytes(_cache()), 0

    def refused(code, f, *a):
        with pytest.raises(fa.FAError) as e:
            f(*a, st)
        assert e.value.code == code

    refused(fa.FA_ERR_INVALID_ARG, fa.fa_cache_append, c, FAKE + 4, FAKE, (128, 64), (128, 64), FAKE, FAKE, 4, fa.FA_BF16)
    refused(fa.FA_ERR_UNSUPPORTED, fa.fa_cache_read, c, FAKE, FAKE, FAKE, 16, fa.FA_FP16)
    refused(fa.FA_ERR_INVALID_ARG, fa.fa_cache_keep, c, FAKE, FAKE + 1, FAKE, 2)
    n = fa.fa_fwd_tree_workspace_bytes(4, 4, 2, 64)
    refused(fa.FA_ERR_WORKSPACE, fa.fa_fwd_tree, c, FAKE, FAKE, FAKE, (256, 64), (256, 64), FAKE, FAKE, None, 0, 4, 4, 2,
            fa.FA_BF16, 0.125, FAKE, n - 1)


@pytest.mark.gpu
def test_python_calls_do_what_the_cache_calls_do():
    from tests.paged import Case, check_attention
    c = Case([20, 3], [2, 3], 2, 64, 16, torch.bfloat16, True, seed=1)
    k, v, q = (x.cuda() for x in (c.new(2), c.new(2), c.new(4)))
    bits = fa.tree_mask([-1, 0, -1, 0, 0], c.cu)
    fa.fa_cache_append(c.cache.args, k, v, k.stride()[:2], v.stride()[:2], c.cu, c.lens, 5, fa.FA_BF16)
    for mask in (None, bits):
        o, lse = torch.empty_like(q), torch.empty(5, 4, device="cuda")
        ws = torch.empty(fa.fa_fwd_tree_workspace_bytes(5, 4, 2, 64), dtype=torch.uint8, device="cuda")
        fa.fa_fwd_tree(c.cache.args, q, o, lse, q.stride()[:2], o.stride()[:2], c.cu, c.lens, mask,
                       0 if mask is None else mask.shape[1], 5, 4, 3, fa.FA_BF16, 0.125, ws, ws.nbytes)
        fa.fa_check_status()
        check_attention(c, q, o, lse, 0.125, mask)
    kept, counts = torch.tensor([[0, 1], [0, 2]], dtype=torch.int32).cuda(), torch.tensor([1, 2], dtype=torch.int32).cuda()
    fa.fa_cache_keep(c.cache.args, c.lens, kept, counts, 2)
    out = [torch.empty(2, 2, 24, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fa.fa_cache_read(c.cache.args, c.lens + counts, *out, 24, fa.FA_BF16)
    fa.fa_check_status()
    for x, y in zip(out, fa.cache_read(c.cache, c.lens + counts, 24)):
        assert torch.equal(x, y)
