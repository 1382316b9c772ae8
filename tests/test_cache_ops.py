"""The calls around the decode step against the fp64 oracle: chunk append, chunk attention, window
decode with weights, eviction; their refusals; and a run of them together.

Tolerances (u = 2**-24, the unit roundoff of fp32; b = 2**-8, that of bf16):
  logits   |dz| <= Z = sigma * sum_c |q_c K_jc| * (d + 4) u * 2: d products accumulated in fp32 (truncated sums
           count twice), one scaling.
  weights  relative error of a softmax weight <= W = 2 (max_j Z + 2**-21): numerator and sum, each with its
           logit's error and that of the exponential (2 units of 2**-22).
  output   <= (W + (n + 64) * 2u) * sum_j p_j |v_j| in fp32: the weights' error and the accumulation of n rows;
           the chunk's weights are rounded to bf16 before the product: + b, and its result to bf16: + b |out|.
"""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as C
from synth import make_problem
from tests.helpers import f64

U, BF = 2.0 ** -24, 2.0 ** -8


def lib_and_session(p, k_max=1, **kw):
    from token_level_sparse_head_b200 import DecodeSession, shape_of

    return DecodeSession(shape_of(p), k_max, device="cuda", dense=kw.pop("dense", False), **kw)


def problem(B, Hq, Hkv, d, seqlens, paged, r=16, seed=3, nan_tail=True, extra_pages=0, **kw):
    """A decode problem whose cache rows behind every sequence are NaN (and infinities)."""
    p = make_problem(B=B, Hq=Hq, Hkv=Hkv, d=d, r=r, seqlens=seqlens, k=1, paged=paged, seed=seed, extra_pages=extra_pages, **kw)
    if nan_tail:
        for b in range(B):
            n = int(p.seqlens[b])
            if paged:
                if n % 64:
                    pg = int(p.page_table[b, n // 64])
                    for x in (p.K, p.V):
                        x[pg, :, n % 64:, ::2] = float("nan")
                        x[pg, :, n % 64:, 1::2] = float("inf")
            else:
                for x in (p.K, p.V):
                    x[b, :, n:, ::2] = float("nan")
                    x[b, :, n:, 1::2] = float("-inf")
    return p


def rows(p, x, b, h, pos):
    pt = None if p.page_table is None else p.page_table.numpy()
    i1, i3 = C.slot(pt, b, pos)
    return f64(x[torch.from_numpy(i1), h, torch.from_numpy(i3)])


def errors_of(q, k, v, sigma, d):
    """(Z per row [G][n], W, sum p |v| [G][d]) of the tolerances above."""
    z = sigma * (np.abs(q) @ np.abs(k).T) * (d + 4) * U * 2
    out, lse, w = C.attend_row(q, k, v, sigma)
    W = 2 * (z.max(axis=1, keepdims=True) + 2.0 ** -21) if k.shape[0] else np.zeros((q.shape[0], 1))
    return out, lse, w, W, w @ np.abs(v)


def starts_of(new):
    return torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)


# ------------------------------------------------------------------------------------ append
APPENDS = [
    # B, Hkv, d, r, seqlens, new, paged, fp8, stride_extra
    (1, 1, 64, 16, [1], [1], False, False, 0),
    (3, 2, 128, 32, [70, 64, 1], [1, 0, 1], True, True, 0),
    (2, 4, 128, 64, [700, 130], [700, 65], True, False, 72),
    (4, 3, 64, 32, [513, 64, 200, 5], [300, 64, 0, 5], False, True, 8),
    (2, 8, 128, 16, [300, 260], [129, 260], False, False, 0),
    (1, 8, 64, 64, [4097], [4001], True, True, 16),
    (2, 8, 128, 32, [2000, 900], [1999, 1], True, False, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hkv,d,r,seqlens,new,paged,fp8,extra", APPENDS)
def test_append_chunk(cuda_lib, B, Hkv, d, r, seqlens, new, paged, fp8, extra):
    p = problem(B, Hkv * 2, Hkv, d, seqlens, paged, r=r, kproj_fp8=fp8, nan_tail=False)
    pad = 3
    n_new = sum(new) + pad
    g = torch.Generator().manual_seed(5)
    buf = torch.randn(n_new, 2 * Hkv * d + extra, generator=g).to(torch.bfloat16)
    k_new, v_new = (buf[:, i * Hkv * d:(i + 1) * Hkv * d].unflatten(1, (Hkv, d)) for i in (0, 1))
    start = starts_of(new)
    pt = None if p.page_table is None else p.page_table.numpy()
    K_ref, V_ref = C.append_chunk(f64(p.K), f64(p.V), f64(k_new), f64(v_new), start.numpy(), seqlens, pt)
    c = p.to("cuda")
    s = lib_and_session(c)
    kp = torch.zeros(*p.K.shape[:3], r, dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16, device="cuda")
    mark = 0x55 if fp8 else 1.0
    (kp.view(torch.uint8) if fp8 else kp).fill_(mark)
    buf_d = buf.cuda()
    kd, vd = (buf_d[:, i * Hkv * d:(i + 1) * Hkv * d].unflatten(1, (Hkv, d)) for i in (0, 1))
    s.append_chunk(kd, vd, start.cuda(), c.M, c.K, c.V, kp, c.page_table, c.seqlens)
    assert s.check()[0] == 0
    assert np.array_equal(f64(c.K), K_ref) and np.array_equal(f64(c.V), V_ref)
    # the projected rows are those of the build over the same cache, the others untouched
    want = torch.zeros_like(kp)
    cuda_lib.sas_build_proj_cache(s.shape, c.K, c.M, want, c.page_table, c.seqlens)
    (want8, kp8) = (want.view(torch.uint8).cpu(), kp.view(torch.uint8).cpu())
    fresh = torch.zeros(kp8.shape[:3], dtype=torch.bool)
    for b in range(B):
        i1, i3 = C.slot(pt, b, np.arange(seqlens[b] - new[b], seqlens[b]))
        fresh[torch.from_numpy(i1), :, torch.from_numpy(i3)] = True
    assert torch.equal(kp8[fresh], want8[fresh])
    untouched = torch.zeros_like(kp)
    (untouched.view(torch.uint8) if fp8 else untouched).fill_(mark)
    assert torch.equal(kp8[~fresh], untouched.view(torch.uint8).cpu()[~fresh])
    # without a projected cache
    K0 = c.K.clone()
    s.append_chunk(kd, vd, start.cuda(), None, c.K, c.V, None, c.page_table, c.seqlens)
    assert torch.equal(K0.view(torch.int16), c.K.view(torch.int16))


@pytest.mark.gpu
def test_append_chunk_one_token_is_append_proj(cuda_lib):
    p = problem(5, 4, 2, 128, [1, 64, 65, 777, 300], True, r=32, nan_tail=False).to("cuda")
    s = lib_and_session(p)
    k_new = torch.randn(5, 2, 128, device="cuda").to(torch.bfloat16)
    a = torch.zeros(*p.K.shape[:3], 32, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros_like(a)
    cuda_lib.sas_append_proj(s.shape, k_new, p.M, a, p.page_table, p.seqlens)
    s.append_chunk(k_new, k_new, torch.arange(6, dtype=torch.int32, device="cuda"), p.M, p.K, p.V, b, p.page_table, p.seqlens)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


# ------------------------------------------------------------------------------------ chunk attention
CHUNKS = [
    # B, Hq, Hkv, d, seqlens, new, paged, window, sinks, pad, fused
    (1, 1, 1, 64, [1], [1], False, 0, 0, 0, False),
    (1, 1, 1, 128, [130], [130], False, 0, 0, 0, False),
    (3, 8, 2, 128, [70, 64, 1], [1, 0, 1], True, 0, 0, 2, True),
    (2, 32, 8, 128, [1500, 333], [5, 5], True, 0, 0, 0, False),
    (2, 8, 2, 64, [700, 129], [700, 65], False, 0, 0, 3, True),
    (4, 6, 2, 128, [513, 64, 200, 5], [300, 64, 0, 5], True, 100, 4, 1, False),
    (2, 10, 2, 64, [515, 260], [40, 260], True, 64, 70, 0, True),
    (2, 20, 4, 128, [900, 77], [101, 77], False, 1, 0, 0, False),
    (3, 16, 1, 128, [2100, 40, 1000], [30, 40, 9], True, 500, 130, 7, False),
    (1, 128, 1, 64, [300], [9], True, 0, 3, 0, False),
    (2, 24, 8, 128, [1000, 640], [600, 640], False, 1 << 30, 5, 0, True),
    (1, 4, 4, 64, [5000], [1024], True, 0, 0, 0, False),
    (1, 8, 2, 128, [9000], [260], False, 2000, 4, 0, False),
]


def check_chunk(p, q, out, lse, out0, new, window, sinks):
    G, sigma, at = p.Hq // p.Hkv, p.d ** -0.5, 0
    out, q = f64(out), f64(q)
    lse = None if lse is None else f64(lse)
    for b in range(p.B):
        n, T = int(p.seqlens[b]), new[b]
        for h in range(p.Hkv):
            k, v = (rows(p, x, b, h, np.arange(n)) for x in (p.K, p.V))
            for t in sorted(set(range(min(T, 40))) | set(range(0, T, 7)) | set(range(max(0, T - 40), T))):
                pos = np.nonzero(C.visible(n - T + t, n, window, sinks))[0]
                ro, rl, w, W, pv = errors_of(q[at + t, h * G:(h + 1) * G], k[pos], v[pos], sigma, p.d)
                o = out[at + t, h * G:(h + 1) * G]
                tol = (W + (len(pos) + 64) * 2 * U + BF) * pv + BF * np.abs(ro) + 1e-30
                assert np.all(np.abs(o - ro) <= tol), (b, h, t, np.max(np.abs(o - ro) / tol))
                if lse is not None:
                    g = lse[at + t, h * G:(h + 1) * G]
                    assert np.all(np.abs(g - rl) <= W[:, 0] + 2.0 ** -21 * (1 + np.abs(rl))), (b, h, t)
        at += T
    assert np.array_equal(out[at:], out0[at:])  # rows behind the last sequence stay as they were


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,d,seqlens,new,paged,window,sinks,pad,fused", CHUNKS)
def test_chunk_attention(cuda_lib, B, Hq, Hkv, d, seqlens, new, paged, window, sinks, pad, fused):
    p = problem(B, Hq, Hkv, d, seqlens, paged)
    c = p.to("cuda")
    for b in range(B):  # what no token of the chunk sees: pages given away, rows that are not finite
        n, T = seqlens[b], new[b]
        seen = np.zeros(n, bool)
        for t in range(T):
            seen |= C.visible(n - T + t, n, window, sinks)
        if T == 0:
            continue
        for x in (c.K, c.V):
            i1, i3 = C.slot(None if p.page_table is None else p.page_table.numpy(), b, np.nonzero(~seen)[0])
            x[torch.from_numpy(i1).cuda(), :, torch.from_numpy(i3).cuda()] = float("nan")
        if paged:
            for lp in range((n + 63) // 64):
                if not seen[lp * 64:lp * 64 + 64].any():
                    c.page_table[b, lp] = -77
    total = sum(new) + pad
    g = torch.Generator().manual_seed(6)
    buf = torch.randn(total, Hq * d + (24 if fused else 0), generator=g).to(torch.bfloat16)
    buf[sum(new):] = float("nan")
    q = buf[:, :Hq * d].unflatten(1, (Hq, d))
    s = lib_and_session(c, chunk=total)
    out = torch.full((total, Hq, d), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((total, Hq), 7.0, device="cuda")
    s.chunk(buf.cuda()[:, :Hq * d].unflatten(1, (Hq, d)), starts_of(new).cuda(), c.K, c.V, c.page_table, c.seqlens,
            window, sinks, out=out, lse=lse)
    assert s.check()[0] == 0
    check_chunk(p, q, out, lse, np.full(out.shape, 7.0), new, window, sinks)
    again, none = s.chunk(q.cuda(), starts_of(new).cuda(), c.K, c.V, c.page_table, c.seqlens, window, sinks)
    assert none is None and torch.equal(again[:sum(new)], out[:sum(new)])


# ------------------------------------------------------------------------------------ window decode
WINDOWS = [
    # B, Hq, Hkv, d, seqlens, paged, window, sinks
    (1, 4, 1, 64, [1], False, 0, 0),
    (4, 8, 2, 128, [0, 1, 64, 65], True, 0, 0),
    (3, 4, 4, 128, [700, 63, 129], True, 100, 4),
    (2, 32, 2, 128, [1000, 333], True, 256, 70),
    (2, 10, 2, 64, [515, 64], False, 1, 0),
    (2, 17, 1, 128, [200, 5], True, 64, 64),
    (1, 40, 1, 64, [999], False, 130, 1000),
    (3, 24, 8, 128, [3000, 100, 2048], True, 1 << 30, 5),
    (2, 64, 8, 128, [5000, 4097], False, 4096, 4),
    (1, 3, 3, 64, [20000], True, 0, 3),
]


def check_window(p, out, lse, acc, acc0, window, sinks):
    G, sigma = p.Hq // p.Hkv, p.d ** -0.5
    for b in range(p.B):
        n = int(p.seqlens[b])
        for h in range(p.Hkv):
            pos = np.nonzero(C.visible(n - 1, n, window, sinks))[0]
            q = f64(p.q[b, h * G:(h + 1) * G])
            k, v = rows(p, p.K, b, h, pos), rows(p, p.V, b, h, pos)
            ro, rl, w, W, pv = errors_of(q, k, v, sigma, p.d)
            o = f64(out[b, h * G:(h + 1) * G])
            tol = (W + (len(pos) + 64) * 2 * U) * pv + 1e-30
            assert np.all(np.abs(o - ro) <= tol), (b, h, np.max(np.abs(o - ro) / tol))
            l = f64(lse[b, h * G:(h + 1) * G])
            if n == 0:
                assert np.all(l == -np.inf)
            else:
                assert np.all(np.abs(l - rl) <= W[:, 0] + 2.0 ** -21 * (1 + np.abs(rl))), (b, h)
            if acc is not None:
                got, was = f64(acc[b, h]), f64(acc0[b, h])
                want = was.copy()
                want[pos] += w.sum(axis=0)
                tol = np.zeros_like(want)
                # one more logit difference, z - log-sum, then G additions
                tol[pos] = 2 * (w * (W + 2.0 ** -21 * (1 + np.abs(rl[:, None])))).sum(axis=0) + (G + 1) * U * want[pos]
                assert np.all(np.abs(got - want) <= tol), (b, h, np.max(np.abs(got - want)))


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,d,seqlens,paged,window,sinks", WINDOWS)
def test_window_decode(cuda_lib, B, Hq, Hkv, d, seqlens, paged, window, sinks):
    p = problem(B, Hq, Hkv, d, seqlens, paged)
    c = p.to("cuda")
    if paged:  # pages that nobody sees may have been given away
        for b in range(B):
            for lp in range((seqlens[b] + 63) // 64):
                pos = np.arange(lp * 64, min(lp * 64 + 64, seqlens[b]))
                if not C.visible(seqlens[b] - 1, seqlens[b], window, sinks)[pos].any():
                    c.page_table[b, lp] = -77
    s = lib_and_session(c, window=True, weights=True)
    acc0 = torch.rand(B, Hkv, p.cap)
    for weights in (False, True):
        acc = acc0.cuda() if weights else None
        out = torch.full((B, Hq, d), 7.0, device="cuda")
        lse = torch.full((B, Hq), 7.0, device="cuda")
        s.window(c.q, c.K, c.V, c.page_table, c.seqlens, window, sinks, weights=acc, out=out, lse=lse)
        assert s.check()[0] == 0
        check_window(p, out, lse, acc, acc0, window, sinks)


@pytest.mark.gpu
def test_window_decode_without_window_is_dense(cuda_lib):
    p = make_problem(B=3, Hq=8, Hkv=2, d=128, r=16, seqlens=[900, 64, 3001], k=1, paged=True, seed=4).to("cuda")
    s = lib_and_session(p, dense=True, window=True)
    a = s.dense(p.q, p.K, p.V, p.page_table, p.seqlens, out=torch.empty(3, 8, 128, device="cuda"))
    b, _ = s.window(p.q, p.K, p.V, p.page_table, p.seqlens, 0, out=torch.empty(3, 8, 128, device="cuda"))
    assert (a - b).abs().max() < 1e-5


@pytest.mark.gpu
def test_window_decode_bad_values_are_reported(cuda_lib):
    p = make_problem(B=2, Hq=4, Hkv=2, d=64, r=16, seqlens=[300, 100], k=1, paged=True, seed=4).to("cuda")
    s = lib_and_session(p, window=True)
    good, _ = s.window(p.q, p.K, p.V, p.page_table, p.seqlens, 0, out=torch.empty(2, 4, 64, device="cuda"))
    bad = p.page_table.clone()
    bad[0, 1] = p.num_pages
    out, _ = s.window(p.q, p.K, p.V, bad, p.seqlens, 0, out=torch.empty(2, 4, 64, device="cuda"))
    assert s.check()[1:] == (2, 0)
    assert torch.equal(out[1], good[1])
    lens = torch.tensor([100000, 100], dtype=torch.int32, device="cuda")
    out, _ = s.window(p.q, p.K, p.V, p.page_table, lens, 0, out=torch.empty(2, 4, 64, device="cuda"))
    assert s.check()[1:] == (1, 0)
    assert torch.equal(out[1], good[1]) and torch.equal(out[0], torch.zeros_like(out[0]))
    assert s.check()[0] == 0


# ------------------------------------------------------------------------------------ eviction
EVICTS = [
    # B, Hkv, d, r, seqlens, keep, sinks, recent, paged, fp8, gate, kind
    (1, 1, 64, 16, [1], [1], 0, 0, False, False, False, "heavy"),
    (3, 2, 128, 32, [700, 64, 65], [100, 64, 10], 4, 16, True, False, True, "heavy"),
    (4, 2, 64, 16, [0, 5, 300, 129], [10, 0, 299, 64], 0, 0, True, True, False, "heavy"),
    (2, 3, 128, 64, [1000, 999], [50, 7], 64, 64, False, True, True, "heavy"),       # more forced rows than the budget
    (2, 2, 128, 16, [5000, 300], [1200, -3], 4, 100, False, False, True, "equal"),   # ties
    (2, 2, 64, 64, [6000, 4500], [3000, 4400], 1, 5, True, False, False, "zeros"),   # ties on zero, most rows kept
    (1, 2, 128, 32, [9000], [2500], 4, 32, True, False, True, "odd"),                # NaN, infinities, negative zero
    (1, 8, 128, 32, [40000], [5000], 4, 256, False, True, False, "heavy"),
]


def evict_weights(kind, B, Hkv, cap, g):
    w = torch.randn(B, Hkv, cap, generator=g).mul(2).exp()
    if kind == "equal":
        w = torch.full_like(w, 0.25)
    if kind == "zeros":
        w = torch.where(torch.rand(B, Hkv, cap, generator=g) < 0.7, torch.zeros_like(w), w)
    if kind == "odd":
        u = torch.rand(B, Hkv, cap, generator=g)
        w[u < 0.1] = float("nan")
        w[(u > 0.1) & (u < 0.12)] = float("inf")
        w[(u > 0.2) & (u < 0.9)] = -0.0
        w[(u > 0.9) & (u < 0.91)] = float("-inf")
    return w


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,Hkv,d,r,seqlens,keep,sinks,recent,paged,fp8,gate,kind", EVICTS)
def test_evict(cuda_lib, B, Hkv, d, r, seqlens, keep, sinks, recent, paged, fp8, gate, kind, in_place):
    p = problem(B, Hkv, Hkv, d, seqlens, paged, r=r, kproj_fp8=fp8, nan_tail=False)
    g = torch.Generator().manual_seed(9)
    w = evict_weights(kind, B, Hkv, p.cap, g)
    log_g = -torch.rand(B, Hkv, p.cap, generator=g) if gate else None
    kp = torch.randint(0, 0x78, (*p.K.shape[:3], r * (1 if fp8 else 2)), generator=g, dtype=torch.uint8)
    c = p.to("cuda")
    keep_max = max(1, max(keep))
    s = lib_and_session(c, k_max=keep_max, evict=True)
    wd, kd, gd = w.cuda(), kp.cuda(), None if log_g is None else log_g.cuda()
    idx = torch.full((B, Hkv, keep_max), -9, dtype=torch.int32, device="cuda")
    w_out = wd if in_place else torch.full_like(wd, 5.0)
    lens = c.seqlens.clone()
    l_out = lens if in_place else torch.full_like(lens, -5)
    s.evict(wd, torch.tensor(keep, dtype=torch.int32, device="cuda"), sinks, recent, c.K, c.V, kd, gd, c.page_table, lens,
            idx=idx, weights_out=w_out, seqlens_out=l_out)
    assert s.check()[0] == 0
    pt = None if p.page_table is None else p.page_table.numpy()
    K, V, P = p.K.view(torch.int16).numpy().copy(), p.V.view(torch.int16).numpy().copy(), kp.numpy().copy()
    W = w.numpy().copy() if in_place else np.full(w.shape, 5.0, np.float32)
    Gt = None if log_g is None else log_g.numpy().copy()
    I = np.full((B, Hkv, keep_max), -1, np.int64)
    for b in range(B):
        n = seqlens[b]
        for h in range(Hkv):
            pos = C.evict_positions(w[b, h].numpy(), n, keep[b], sinks, recent)
            m = len(pos)
            I[b, h, :m] = pos
            s1, s3 = C.slot(pt, b, pos)
            d1, d3 = C.slot(pt, b, np.arange(m))
            for x in (K, V, P):
                x[d1, h, d3] = x[s1, h, s3]
            if Gt is not None:
                Gt[b, h, :m] = Gt[b, h, pos]
            W[b, h, :n] = 0.0
            W[b, h, :m] = w[b, h].numpy()[pos]
    assert np.array_equal(idx.cpu().numpy(), I)
    assert l_out.tolist() == [min(n, max(0, k)) for n, k in zip(seqlens, keep)]
    assert np.array_equal(c.K.view(torch.int16).cpu().numpy(), K) and np.array_equal(c.V.view(torch.int16).cpu().numpy(), V)
    assert np.array_equal(kd.cpu().numpy(), P)
    assert np.array_equal(w_out.cpu().numpy(), W, equal_nan=True)
    if gate:
        assert np.array_equal(gd.cpu().numpy(), Gt)


@pytest.mark.gpu
def test_evict_leaves_the_workspace_ready_for_a_decode_step(cuda_lib):
    """The selection's histograms are zero again: a sparse step on the same workspace is unchanged."""
    p = make_problem(B=2, Hq=8, Hkv=2, d=128, r=32, seqlens=[3000, 515], k=[200, 100], k_max=600, paged=True, seed=21).to("cuda")
    s = lib_and_session(p, k_max=600, evict=True)
    kp = torch.zeros(*p.K.shape[:3], 32, dtype=torch.bfloat16, device="cuda")
    cuda_lib.sas_build_proj_cache(s.shape, p.K, p.M, kp, p.page_table, p.seqlens)
    a, ia = (t.clone() for t in s.decode(p.q, p.M, kp, p.K, p.V, p.page_table, p.seqlens, p.k))
    w = torch.rand(2, 2, p.cap, device="cuda")
    s.evict(w, torch.tensor([500, 600], dtype=torch.int32, device="cuda"), 4, 8, p.K.clone(), p.V.clone(), None, None,
            p.page_table, p.seqlens, idx=torch.empty(2, 2, 600, dtype=torch.int32, device="cuda"), weights_out=w.clone(),
            seqlens_out=p.seqlens.clone())
    b, ib = s.decode(p.q, p.M, kp, p.K, p.V, p.page_table, p.seqlens, p.k)
    assert torch.equal(ia, ib) and torch.equal(a, b) and s.check()[0] == 0
