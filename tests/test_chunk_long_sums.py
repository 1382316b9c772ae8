"""Chunk attention over long caches: what the sums of a hundred thousand rows are off by.

The matrix instruction truncates.  A step adds 16 products to the running output; if each of the 17
terms loses up to 2^-25 of the result, a step is off by 17 * 2^-25 and always towards zero.  Over K
steps of equal weights the running output grows evenly, so the sum is off by K / 2 * 17 * 2^-25 of
itself: 2.6e-4 for the 1024 steps after which the kernel adds its output to a sum with rounding (whose
additions, and the division, are off by less than 2^-19), and 4e-3 for the 16384 steps of 262144 rows.
"""
import numpy as np
import pytest
import torch

from tests.helpers import f64
from tests.test_cache_ops import BF, U, errors_of
from token_level_sparse_head_b200 import DecodeSession, Shape

CAP = 262144


def session(B, Hq, d, T, paged):
    shape = Shape(B, Hq, 1, d, 16, 0, 64, CAP // 64, CAP // 64) if paged else Shape(B, Hq, 1, d, 16, CAP)
    return DecodeSession(shape, 1, dense=False, chunk=T)


CASES = [
    # B, Hq, d, new tokens a sequence, paged: every CTA has a task of its own, or several whole ones
    (1, 1, 128, 37888, False),     # two tiles a task, 2048 units of 128 keys
    (1, 2, 64, 18944, False),
    (148, 32, 128, 4, True),       # one tile: two warpgroups, 1024 units of 256 keys
    (148, 3, 64, 42, True),        # with rows that no token fills
]


def caches(B, d, paged, K, V):
    """K, V [CAP][d] as the cache of every sequence (paged: all of them read the same pages)."""
    if not paged:
        return K.view(1, 1, CAP, d).contiguous(), V.view(1, 1, CAP, d).contiguous(), None
    table = torch.randperm(CAP // 64, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    x = [torch.empty(CAP // 64, 1, 64, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for c, y in zip(x, (K, V)):
        c[table.long().cuda()] = y.view(CAP // 64, 1, 64, d)
    return x[0], x[1], table.cuda().expand(B, -1).contiguous()


def run(B, Hq, d, T, paged, K, V, q):
    s = session(B, Hq, d, B * T, paged)
    k, v, table = caches(B, d, paged, K, V)
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda") * T
    lse = torch.empty(B * T, Hq, device="cuda")
    out, _ = s.chunk(q, start, k, v, table, torch.full((B,), CAP, dtype=torch.int32, device="cuda"), lse=lse)
    assert s.check()[0] == 0
    return out, lse


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,d,T,paged", CASES)
def test_equal_weights(cuda_lib, B, Hq, d, T, paged):
    """Every weight is 1, so nothing but the sums of V, the division and the result's rounding can be off.
    V's values lie over 2^-8 .. 2, so that a sum has bits to lose from its first block on."""
    g = torch.Generator(device="cuda").manual_seed(3)
    V = (1 + torch.rand(CAP, d, generator=g, device="cuda")) * 2.0 ** -torch.randint(0, 8, (CAP, d), generator=g, device="cuda")
    V = (V * (1 + torch.rand(d, generator=g, device="cuda"))).to(torch.bfloat16)
    K = torch.zeros(CAP, d, dtype=torch.bfloat16, device="cuda")
    q = torch.randn(B * T, Hq, d, device="cuda").to(torch.bfloat16)
    out, lse = run(B, Hq, d, T, paged, K, V, q)
    seen = torch.arange(CAP - T + 1, CAP + 1, device="cuda")
    mean = V[:CAP - T].double().sum(0) + V[CAP - T:].double().cumsum(0)
    mean = (mean / seen[:, None].double()).repeat(B, 1)[:, None]
    half = torch.exp2(torch.floor(torch.log2(mean)) - 8)  # half a step of bf16
    off = (out.double() - mean).abs()
    assert (off <= half + 3e-4 * mean).all(), ((off - half) / mean).max()
    log = seen.double().log().repeat(B)[:, None]
    assert ((lse.double() - log).abs() <= 2.0 ** -21 * (1 + log)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,d,T,paged", CASES)
@pytest.mark.parametrize("rise", [-24.0, 24.0])
def test_weights_that_rise_or_fall_along_the_cache(cuda_lib, B, Hq, d, T, paged, rise):
    """The running maximum moves all the way (or stands from the first block on) while sums are put aside."""
    g = torch.Generator(device="cuda").manual_seed(4)
    K = torch.randn(CAP, d, generator=g, device="cuda") * 0.5
    K[:, 0] = torch.linspace(0, rise, CAP, device="cuda") * d ** 0.5
    V = (torch.rand(CAP, d, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    K = K.to(torch.bfloat16)
    q = torch.randn(B * T, Hq, d, generator=g, device="cuda")
    q[:, :, 0] = 1
    q = q.to(torch.bfloat16)
    out, lse = run(B, Hq, d, T, paged, K, V, q)
    k, v = f64(K), f64(V)
    for b, t in ((0, 0), (0, T - 1), (B // 2, T // 2), (B - 1, T - 1)):
        n = CAP - T + t + 1
        qt = f64(q[b * T + t])
        ro, rl, _, W, pv = errors_of(qt, k[:n], v[:n], d ** -0.5, d)
        tol = (W + 3e-4 + BF) * pv + BF * np.abs(ro)
        assert np.all(np.abs(f64(out[b * T + t]) - ro) <= tol), (b, t)
        assert np.all(np.abs(f64(lse[b * T + t]) - rl) <= W[:, 0] + 2.0 ** -21 * (1 + np.abs(rl))), (b, t)
