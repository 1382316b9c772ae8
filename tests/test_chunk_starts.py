"""Chunk batches whose q_start is out of order or range: which sequences are skipped, and that the
others are as if those were not there.  Tolerances as derived in tests/test_cache_ops.py.
"""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as C
from synth import make_problem
from tests.helpers import f64
from token_level_sparse_head_b200 import lib as L
from tests.test_cache_ops import BF, U, errors_of, lib_and_session, rows

LENS, NEW = [300, 100, 200, 50], 40
LOW, HIGH = -2 ** 31, 2 ** 31 - 1
STARTS = [
    # q_start, seqlens, codes
    ([0, 10, 20, 30, 40], LENS, [0, 0, 0, 0]),
    ([3, 3, 20, 20, 33], LENS, [0, 0, 0, 0]),              # rows that belong to nobody around and nobody's
    ([0, 10, 5, 40, 40], LENS, [0, 6, 6, 0]),              # a fall, and a start below the end before it
    ([0, 40, 0, 40, 40], LENS, [0, 6, 6, 0]),              # the same rows twice
    ([10, 5, 20, 30, 40], LENS, [6, 6, 0, 0]),
    ([0, 41, 20, 30, 40], LENS, [6, 6, 6, 6]),             # an entry past the arrays: the rest lies below it
    ([0, 10, 20, 50, 60], LENS, [0, 0, 6, 6]),             # the last one wholly past them
    ([-3, 10, 20, 30, 40], LENS, [6, 0, 0, 0]),
    ([-9, -3, 20, 30, 40], LENS, [6, 6, 0, 0]),
    ([LOW, HIGH, LOW, HIGH, 0], LENS, [6, 6, 6, 6]),
    ([0, 10, 10, 30, 40], [300, -1, 200, 50], [0, 1, 0, 0]),      # a bad length without new tokens
    ([0, 10, 20, 30, 40], [300, 100, 1 << 30, 50], [0, 0, 1, 0]),
    ([0, 10, 20, 30, 40], [9, 100, 200, 50], [6, 0, 0, 0]),       # more new tokens than cached ones
]


@pytest.mark.parametrize("start,lens,codes", STARTS)
def test_which_sequences_are_skipped(start, lens, codes):
    assert C.chunk_errors(start, lens, NEW, 320) == codes
    taken = [(start[b], start[b + 1]) for b in range(4) if codes[b] == 0]
    assert all(a[1] <= b[0] for a, b in zip(taken, taken[1:]))  # none shares a row


def check_outputs(p, q, start, lens, codes, out, lse):
    G, sigma = p.Hq // p.Hkv, p.d ** -0.5
    out, lse, q = f64(out), f64(lse), f64(q)
    left = np.ones(out.shape[0], bool)
    for b, why in enumerate(codes):
        if why:
            continue
        n, s0, s1 = lens[b], start[b], start[b + 1]
        left[s0:s1] = False
        for h in range(p.Hkv):
            k, v = (rows(p, x, b, h, np.arange(n)) for x in (p.K, p.V))
            for t in range(s0, s1):
                m = n - (s1 - s0) + (t - s0) + 1
                ro, rl, _, W, pv = errors_of(q[t, h * G:(h + 1) * G], k[:m], v[:m], sigma, p.d)
                tol = (W + (m + 64) * 2 * U + BF) * pv + BF * np.abs(ro) + 1e-30
                assert np.all(np.abs(out[t, h * G:(h + 1) * G] - ro) <= tol), (b, h, t)
                assert np.all(np.abs(lse[t, h * G:(h + 1) * G] - rl) <= W[:, 0] + 2.0 ** -21 * (1 + np.abs(rl)))
    assert np.all(out[left] == 7.0) and np.all(lse[left] == 7.0)


@pytest.mark.gpu
@pytest.mark.parametrize("start,lens,codes", STARTS)
def test_chunk_attention_skips(cuda_lib, start, lens, codes):
    p = make_problem(B=4, Hq=4, Hkv=2, d=64, r=16, seqlens=LENS, k=1, paged=True, seed=4)
    c = p.to("cuda")
    s = lib_and_session(c, chunk=64)
    q = torch.randn(NEW, 4, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    out = torch.full((NEW, 4, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((NEW, 4), 7.0, device="cuda")
    s.chunk(q.cuda(), torch.tensor(start, dtype=torch.int32, device="cuda"), c.K, c.V, c.page_table,
            torch.tensor(lens, dtype=torch.int32, device="cuda"), out=out, lse=lse)
    status, code, where = s.check()
    assert code == max(codes) and (code == 0 or codes[where] == code)
    check_outputs(p, q, start, lens, codes, out, lse)


def many(most=5, B=1500):
    """More sequences than a CTA has threads, some of them malformed."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(1, 60, B)]
    new = [int(min(n, x)) for n, x in zip(lens, rng.integers(0, most + 1, B))]
    start = [0] + [int(x) for x in np.cumsum(new)]
    total = start[-1]
    start[700] = start[700] + 9            # above its successors
    start[1200] = start[1100]              # a start below earlier ones
    start[1400] = total + 1                # past the arrays, the rest below it
    return lens, start, total


@pytest.mark.gpu
def test_chunk_attention_skips_in_a_large_batch(cuda_lib):
    lens, start, total = many()
    p = make_problem(B=len(lens), Hq=2, Hkv=1, d=64, r=16, seqlens=lens, k=1, paged=True, seed=3)
    codes = C.chunk_errors(start, lens, total, p.cap)
    assert codes.count(6) > 100 and codes.count(0) > 1300
    c = p.to("cuda")
    s = lib_and_session(c, chunk=total)
    q = torch.randn(total, 2, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    out = torch.full((total, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((total, 2), 7.0, device="cuda")
    s.chunk(q.cuda(), torch.tensor(start, dtype=torch.int32, device="cuda"), c.K, c.V, c.page_table, c.seqlens, out=out, lse=lse)
    assert s.check()[1] == 6
    check_outputs(p, q, start, lens, codes, out, lse)


def run_append(p, start, lens, n_new, with_proj):
    """Appends into copies of the caches and checks every row: those of taken sequences, and no other."""
    c = p.to("cuda")
    s = lib_and_session(c)
    g = torch.Generator().manual_seed(6)
    kn, vn = (torch.randn(n_new, p.Hkv, p.d, generator=g).to(torch.bfloat16) for _ in range(2))
    kp = torch.full((*p.K.shape[:3], p.r), 7.0, dtype=torch.bfloat16, device="cuda") if with_proj else None
    s.append_chunk(kn.cuda(), vn.cuda(), torch.tensor(start, dtype=torch.int32, device="cuda"), c.M, c.K, c.V, kp, c.page_table,
                   torch.tensor(lens, dtype=torch.int32, device="cuda"))
    report = s.check()
    codes = C.chunk_errors(start, lens, n_new, p.cap)
    pt = None if p.page_table is None else p.page_table.numpy()
    K, V, fresh = f64(p.K), f64(p.V), torch.zeros(p.K.shape[:3], dtype=torch.bool)
    for b, why in enumerate(codes):
        if why == 0 and start[b + 1] > start[b]:
            i1, i3 = C.slot(pt, b, np.arange(lens[b] - (start[b + 1] - start[b]), lens[b]))
            K[i1, :, i3], V[i1, :, i3] = f64(kn[start[b]:start[b + 1]]), f64(vn[start[b]:start[b + 1]])
            fresh[torch.from_numpy(i1), :, torch.from_numpy(i3)] = True
    assert np.array_equal(f64(c.K), K) and np.array_equal(f64(c.V), V)
    if with_proj:  # the projected rows are the build's over the same rows
        want = torch.zeros_like(kp)
        s_lens = torch.tensor([min(max(n, 0), p.cap) for n in lens], dtype=torch.int32, device="cuda")
        L.sas_build_proj_cache(s.shape, c.K, c.M, want, c.page_table, s_lens)
        got = kp.cpu()
        assert torch.equal(got[fresh], want.cpu()[fresh]) and (got[~fresh] == 7.0).all()
    return codes, report


@pytest.mark.gpu
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("Hkv,d", [(2, 64), (56, 128)])   # a CTA per token and head; tiles of tokens
@pytest.mark.parametrize("start,lens,codes", STARTS)
def test_append_skips(cuda_lib, start, lens, codes, Hkv, d, paged):
    p = make_problem(B=4, Hq=Hkv, Hkv=Hkv, d=d, r=16, seqlens=LENS, k=1, paged=paged, seed=4)
    for with_proj in (False, True):
        got, (status, code, where) = run_append(p, start, lens, NEW, with_proj)
        assert got == codes and code == max(codes) and (code == 0 or codes[where] == code)


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,most", [(1, 1), (2, 5)])   # a CTA per token and head; tiles of tokens
def test_append_skips_in_a_large_batch(cuda_lib, Hkv, most):
    lens, start, total = many(most)
    p = make_problem(B=len(lens), Hq=Hkv, Hkv=Hkv, d=64, r=16, seqlens=lens, k=1, paged=True, seed=3)
    codes, report = run_append(p, start, lens, total, True)
    assert report[1] == 6 and codes.count(6) > 100


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv", [2, 56])
def test_append_reports_a_page_outside_the_cache(cuda_lib, Hkv):
    p = make_problem(B=4, Hq=Hkv, Hkv=Hkv, d=64, r=16, seqlens=LENS, k=1, paged=True, seed=4)
    c = p.to("cuda")
    s = lib_and_session(c)
    c.page_table[2, 3] = p.num_pages
    x = torch.randn(NEW, Hkv, 64, device="cuda").to(torch.bfloat16)
    K = c.K.clone()
    s.append_chunk(x, x, torch.tensor([0, 10, 20, 30, 40], dtype=torch.int32, device="cuda"), None, K, c.V, None, c.page_table, c.seqlens)
    assert s.check()[1:] == (2, 2)
    for b, (n, t0) in enumerate(zip(LENS, (0, 10, 20, 30))):
        for t in range(10):
            pos = n - 10 + t
            pg = int(p.page_table[b, pos // 64])
            good = b != 2 or pos // 64 != 3
            assert torch.equal(K[pg, :, pos % 64], x[t0 + t] if good else c.K[pg, :, pos % 64])
