"""The calls around the step at the ends of their ranges: the most new tokens, the most sequences, budgets
above the capacity, windows, sinks and newest rows as large as an int holds.

Tolerances as derived in tests/test_cache_ops.py, with a bound on a logit's error for all rows: sigma sum |q_c K_c|
<= |q| |K| / 8 stays below 18 for normal rows of 64 channels, so Z <= 18 * 68 * 2 u = 1.5e-4 and W = 2 Z = 3e-4;
with K scaled by 0.3 W = 1e-4.
"""
import pytest
import torch

from oracle import cache_oracle as C
from tests.test_cache_ops import BF
from token_level_sparse_head_b200 import DecodeSession, Shape

BIG = 2 ** 31 - 1


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bf16(*shape, seed=1, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * scale).to(torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("keep,sinks,recent", [(500, 0, 0), (70, BIG, 0), (70, 0, BIG), (70, 5, BIG), (70, BIG, BIG), (0, 3, 3)])
def test_evict_budgets_and_forced_rows(cuda_lib, keep, sinks, recent):
    """idx_out is wider than the cache has rows."""
    lens, cap = [130, 77], 132
    K, V, w = bf16(2, 2, cap, 64), bf16(2, 2, cap, 64, seed=2), torch.rand(2, 2, cap, device="cuda")
    s = DecodeSession(Shape(2, 2, 2, 64, 16, cap), 500, dense=False, evict=True)
    K0, V0, kept = K.clone(), V.clone(), torch.zeros(2, dtype=torch.int32, device="cuda")
    idx = s.evict(w, i32([keep, keep]), sinks, recent, K, V, None, None, None, i32(lens), weights_out=torch.empty_like(w), seqlens_out=kept)
    assert s.check()[0] == 0 and kept.tolist() == [min(n, keep) for n in lens]
    for b, n in enumerate(lens):
        for h in range(2):
            pos = C.evict_positions(w[b, h].cpu().numpy(), n, keep, min(sinks, n), recent).tolist()
            m = len(pos)
            assert idx[b, h, :m].tolist() == pos and (idx[b, h, m:] == -1).all()
            for x, x0 in ((K, K0), (V, V0)):
                assert torch.equal(x[b, h, :m], x0[b, h, pos]) and torch.equal(x[b, h, m:], x0[b, h, m:])


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(BIG, 0), (BIG, BIG), (1, BIG), (700, 0), (0, BIG), (-5, 7)])
def test_windows_that_hide_nothing(cuda_lib, window, sinks):
    """The pages are the same, in the same order, so the results are the same bits."""
    n, T = 700, 90
    K, V, q, start, lens = bf16(1, 1, n, 64), bf16(1, 1, n, 64, seed=2), bf16(T, 4, 64, seed=3), i32([0, T]), i32([n])
    s = DecodeSession(Shape(1, 4, 1, 64, 16, n), 1, dense=False, chunk=T, window=True)
    want, _ = s.chunk(q, start, K, V, None, lens)
    want1 = s.window(q[-1:], K, V, None, lens, 0)[0].clone()
    got, _ = s.chunk(q, start, K, V, None, lens, window, sinks)
    got1, _ = s.window(q[-1:], K, V, None, lens, window, sinks)
    assert s.check()[0] == 0
    if window == 1:  # its pages are listed as sinks and window: other shares
        assert (got.float() - want.float()).abs().max() <= 4 * BF and (got1 - want1).abs().max() < 1e-5
    else:
        assert torch.equal(got, want) and torch.equal(got1, want1)


@pytest.mark.gpu
def test_the_most_new_tokens(cuda_lib):
    B, cap = 16, 262144
    T = B * cap
    K, V, q = bf16(B, 1, cap, 64, scale=0.3), bf16(B, 1, cap, 64, seed=2), bf16(T, 1, 64, seed=3)
    start, lens = torch.arange(B + 1, device="cuda", dtype=torch.int32) * cap, i32([cap] * B)
    s = DecodeSession(Shape(B, 1, 1, 64, 16, cap), 1, dense=False, chunk=T)
    lse = torch.empty(T, 1, device="cuda")
    out, _ = s.chunk(q, start, K, V, None, lens, lse=lse)
    assert T == 1 << 22 and s.check()[0] == 0
    for b, t in ((0, 0), (0, 1), (3, 100000), (7, 262143), (15, 200001), (15, 262143)):
        z = (K[b, 0, :t + 1].double() @ q[b * cap + t, 0].double()) / 8
        p, v = torch.softmax(z, 0), V[b, 0, :t + 1].double()
        # with the sums' 3e-4 of tests/test_chunk_long_sums.py
        assert ((out[b * cap + t, 0].double() - p @ v).abs() <= BF * (p @ v).abs() + (BF + 4e-4) * (p @ v.abs())).all(), (b, t)
        assert (lse[b * cap + t, 0].double() - torch.logsumexp(z, 0)).abs() <= 1e-4 + 2.0 ** -21 * 16
    s.append_chunk(q, q, start, None, K, V, None, None, lens)
    assert s.check()[0] == 0 and torch.equal(K.view(T, 1, 64), q) and torch.equal(V.view(T, 1, 64), q)


@pytest.mark.gpu
def test_the_most_sequences(cuda_lib):
    B = 65535
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 65, (B,), generator=g)
    new = torch.minimum(lens, torch.randint(0, 3, (B,), generator=g))
    table = torch.randperm(B, generator=g).int().view(B, 1).cuda()
    T = int(new.sum())
    start = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).cuda()
    K, V, rows, q, q1 = bf16(B, 1, 64, 64), bf16(B, 1, 64, 64, seed=2), bf16(T, 1, 64, seed=3), bf16(T, 2, 64, seed=4), bf16(B, 2, 64, seed=5)
    n, st = lens.int().cuda(), start.int()
    s = DecodeSession(Shape(B, 2, 1, 64, 16, 0, 64, 1, B), 20, dense=False, chunk=T, window=True, weights=True, evict=True)
    s.append_chunk(rows, rows, st, None, K, V, None, table, n)
    b = torch.repeat_interleave(torch.arange(B), new).cuda()
    pos = lens.cuda()[b] - new.cuda()[b] + torch.arange(T, device="cuda") - start[b]
    assert torch.equal(K[table[b, 0].long(), 0, pos], rows[:, 0])
    k, v = (x[table[:, 0].long(), 0].double() for x in (K, V))
    out, _ = s.chunk(q, st, K, V, table, n)
    z = torch.einsum("thd,tnd->thn", q.double(), k[b]) / 8
    p = torch.softmax(z.masked_fill(torch.arange(64, device="cuda") > pos[:, None, None], -1e300), -1)
    ref, size = p @ v[b], p @ v[b].abs()
    assert ((out.double() - ref).abs() <= BF * ref.abs() + (BF + 4e-4) * size).all()
    acc = torch.zeros(B, 1, 64, device="cuda")
    one, _ = s.window(q1, K, V, table, n, 0, weights=acc)
    seen = torch.arange(64, device="cuda")[None, None] < n[:, None, None]
    p = torch.softmax((torch.einsum("bhd,bnd->bhn", q1.double(), k) / 8).masked_fill(~seen, -1e300), -1) * seen
    assert ((one.double() - p @ v).abs() <= 4e-4 * (p @ v.abs())).all() and ((acc[:, 0].double() - p.sum(1)).abs() <= 1e-3 * p.sum(1)).all()
    keep, kept = torch.full((B,), 20, dtype=torch.int32, device="cuda"), torch.empty_like(n)
    w = torch.rand(B, 1, 64, device="cuda")
    idx = s.evict(w, keep, 1, 2, K, V, None, None, table, n, weights_out=torch.empty_like(w), seqlens_out=kept)
    assert s.check()[0] == 0 and torch.equal(kept, torch.minimum(n, keep))
    for i in (0, 1, 777, B - 1):
        pos = C.evict_positions(w[i, 0].cpu().numpy(), int(lens[i]), 20, 1, 2).tolist()
        assert idx[i, 0, :len(pos)].tolist() == pos
        assert torch.equal(K[int(table[i, 0]), 0, :len(pos)].double(), k[i, pos])
