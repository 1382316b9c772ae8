"""Chunk attention whose KV heads are gone through in several waves, on both sides of the rule's bounds.

Tolerances as derived in tests/test_cache_ops.py.
"""
import pytest
import torch

from synth import make_problem
from tests.test_cache_ops import lib_and_session, starts_of
from tests.test_cache_ops_together import check_rows


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d,lens,new,paged,window", [
    (32, 8, 128, [33000], [700], True, 0),             # two waves, lists made by the CTAs
    (32, 8, 128, [33000], [300], False, 0),            # the same cache, too few units for more than one
    (32, 8, 128, [70000], [600], False, 0),            # four waves
    (32, 8, 128, [140000], [300], True, 0),
    (12, 4, 64, [90000, 60000], [900, 700], True, 0),  # two sequences of groups of 3
    (16, 2, 128, [90000], [2000], False, 0),           # as many waves as KV heads
    (16, 2, 128, [90000], [2000], False, 50000),
    (10, 5, 128, [40000, 3, 20000], [700, 3, 900], True, 0),  # KV heads that the waves share unevenly
])
def test_waves(cuda_lib, Hq, Hkv, d, lens, new, paged, window):
    p = make_problem(B=len(lens), Hq=Hq, Hkv=Hkv, d=d, r=16, seqlens=lens, k=1, paged=paged, seed=7)
    c = p.to("cuda")
    total = sum(new)
    s = lib_and_session(c, chunk=total)
    q = torch.randn(total, Hq, d, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    lse = torch.full((total, Hq), 7.0, device="cuda")
    out, _ = s.chunk(q.cuda(), starts_of(new).cuda(), c.K, c.V, c.page_table, c.seqlens, window, 4, lse=lse)
    assert s.check()[0] == 0
    tokens = [(b, t) for b, T in enumerate(new) for t in {0, T // 2 + 1, T - 1} if t < T]
    check_rows(p, q, out, lse, new, window, 4, tokens)
    again, _ = s.chunk(q.cuda(), starts_of(new).cuda(), c.K, c.V, c.page_table, c.seqlens, window, 4)
    assert torch.equal(again, out)
