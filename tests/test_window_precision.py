"""The window decode's fp32 outputs: that the weights keep their 24 bits and the sums are rounded; and the
longest list of pages that it can cut into shares.

The bounds here are those of single roundings, not of a whole softmax, so fewer bits anywhere show.
"""
import numpy as np
import pytest
import torch

from tests.helpers import f64
from token_level_sparse_head_b200 import DecodeSession, Shape, lib

U = 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("d,Hq", [(64, 8), (128, 8), (64, 16), (128, 16), (128, 5)])
def test_a_weight_keeps_its_bits(cuda_lib, d, Hq):
    """Two rows count: row 0 with logit 0 and V = 0, row 5 with logit -a, so out = e / (1 + e) * V with e = exp(-a).

    q . K is exact (one product); a log2(e) carries 3 roundings (the scale's two, the product's), so e is off
    by 3 a u and the exponential's 2^-22; the sum, the inverse and three products add 8 u.  a <= 4:
    (12 + 4 + 8) u = 1.5e-6.  A weight of two bf16 terms would be off by up to 2^-17 = 7.6e-6."""
    B, n = 40, 16
    g = torch.Generator().manual_seed(1)
    a = (torch.rand(B, Hq, generator=g) * 3.9 + 0.05) * d ** 0.5
    q = torch.zeros(B, Hq, d)
    q[:, :, 0], q[:, :, 1] = -a, -1024.0
    K, V = torch.zeros(B, 1, 64, d), torch.randn(B, 1, 64, d, generator=g)
    K[:, :, 1:n, 1] = 64.0                      # rows whose weight is 0
    K[:, :, 5, 1], K[:, :, 5, 0] = 0.0, 1.0
    V[:, :, 0] = 0.0
    q, K, V = (x.to(torch.bfloat16) for x in (q, K, V))
    s = DecodeSession(Shape(B, Hq, 1, d, 16, 64), 1, dense=False, window=True)
    out, _ = s.window(q.cuda(), K.cuda(), V.cuda(), None, torch.full((B,), n, dtype=torch.int32, device="cuda"), 0)
    e = np.exp(f64(q)[:, :, 0] * d ** -0.5)[:, :, None]
    want = e / (1 + e) * f64(V)[:, :, 5]
    assert s.check()[0] == 0
    assert np.all(np.abs(f64(out) - want) <= 24 * U * np.abs(want)), np.max(np.abs(f64(out) / want - 1))


@pytest.mark.gpu
@pytest.mark.parametrize("d,Hq", [(64, 8), (128, 8), (128, 16)])
def test_sums_of_many_rows_are_rounded(cuda_lib, d, Hq):
    """Equal weights over 65536 rows of 32 sequences: 222 pages a CTA, 111 of them a warp's.

    A warp adds 111 products of 16 rows; with equal weights the sum grows evenly, so its roundings are off by at most
    111 / 2 u, the joins of 8 warps and of at most 148 / 32 + 2 CTAs by 15 u, and a product of 16 rows, which the
    matrix instruction truncates, by 17 * 2^-25: 79 u = 4.7e-6.  Roundings go up and down alike, so the mean over the
    columns stays near the product's part, at most 8.5 u = 5.1e-7; sums that are truncated each time lie 5e-6 low."""
    B, n = 32, 65536
    g = torch.Generator(device="cuda").manual_seed(3)
    V = (1 + torch.rand(n, d, generator=g, device="cuda")) * 2.0 ** -torch.randint(0, 8, (n, d), generator=g, device="cuda")
    V = (V * (1 + torch.rand(d, generator=g, device="cuda"))).to(torch.bfloat16)
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()  # all sequences read the same pages
    s = DecodeSession(Shape(B, Hq, 1, d, 16, 0, 64, n // 64, n // 64), 1, dense=False, window=True)
    q = torch.randn(B, Hq, d, generator=g, device="cuda").to(torch.bfloat16)
    lse = torch.empty(B, Hq, device="cuda")
    out, _ = s.window(q, torch.zeros(n // 64, 1, 64, d, dtype=torch.bfloat16, device="cuda"), V.view(n // 64, 1, 64, d), table,
                      torch.full((B,), n, dtype=torch.int32, device="cuda"), 0, lse=lse)
    assert s.check()[0] == 0
    off = out.double() / V.double().mean(0) - 1
    assert off.abs().max() <= 79 * U and off.mean().abs() <= 1e-6, (off.abs().max(), off.mean())
    assert (lse.double() - np.log(n)).abs().max() <= 2.0 ** -21 * (1 + np.log(n))


def test_a_list_of_pages_that_32_bits_cannot_share_out():
    """524160 head groups of 4097 pages: 128 below 2^31, where a share rounded up times the last CTA passes it."""
    groups, at = 524160, 1 << 20
    assert 0 < 2 ** 31 - groups * (262144 // 64 + 1) < 148
    shape = Shape(1, 16 * groups, 1, 64, 16, n_cap=262144)
    with pytest.raises(lib.SasError) as e:
        lib.sas_window_decode(shape, at, at, at, None, at, 0, 0, at, at, None, at, 1 << 40, 0)
    assert e.value.status == lib.SAS_ERR_UNSUPPORTED
