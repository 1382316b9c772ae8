"""The calls around the decode step: refusals on the host, values that only the device sees, streams
and graphs, the paths of large batches and caches, and a run of them together.

Tolerances as derived in tests/test_cache_ops.py.
"""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as C
from synth import make_problem
from tests.helpers import f64
from tests.test_cache_ops import BF, U, check_chunk, check_window, errors_of, lib_and_session, problem, rows, starts_of
from token_level_sparse_head_b200 import lib as L

P = 1 << 20  # a 16-byte-aligned dummy address; never dereferenced (validation fails first)


def _expect(status, fn, *args):
    with pytest.raises(L.SasError) as e:
        fn(*args)
    assert e.value.status == status, str(e.value)


# ------------------------------------------------------------------------------------ refusals (host)
SHAPE = L.Shape(2, 8, 2, 64, 16, n_cap=512)
BIG = 1 << 40


def _call(name, shape=SHAPE, **over):
    a = dict(q=P, K_new=P, V_new=P, stride=8 * 64, q_start=P, n_new=9, M=P, K=P, V=P, Kproj=P, page_table=None, seqlens=P,
             window=0, sinks=0, out=P, lse=P, weights=P, keep=P, keep_max=4, recent=0, log_g=P, idx=P, w_out=P, l_out=P,
             ws=P, ws_bytes=BIG)
    a.update(over)
    if name == "append":
        L.sas_append_chunk(shape, a["K_new"], a["V_new"], a["stride"], a["q_start"], a["n_new"], a["M"], a["K"], a["V"],
                           a["Kproj"], a["page_table"], a["seqlens"], a["ws"], a["ws_bytes"], 0)
    elif name == "chunk":
        L.sas_chunk_attention(shape, a["q"], a["stride"], a["q_start"], a["n_new"], a["K"], a["V"], a["page_table"],
                              a["seqlens"], a["window"], a["sinks"], a["out"], a["lse"], a["ws"], a["ws_bytes"], 0)
    elif name == "window":
        L.sas_window_decode(shape, a["q"], a["K"], a["V"], a["page_table"], a["seqlens"], a["window"], a["sinks"], a["out"],
                            a["lse"], a["weights"], a["ws"], a["ws_bytes"], 0)
    else:
        L.sas_evict(shape, a["weights"], a["keep"], a["keep_max"], a["sinks"], a["recent"], a["K"], a["V"], a["Kproj"],
                    a["log_g"], a["page_table"], a["seqlens"], a["idx"], a["w_out"], a["l_out"], a["ws"], a["ws_bytes"], 0)


NEEDED = {"append": ["K_new", "V_new", "q_start", "M", "K", "V", "seqlens"], "chunk": ["q", "q_start", "K", "V", "seqlens", "out", "ws"],
          "window": ["q", "K", "V", "seqlens", "out", "ws"],
          "evict": ["weights", "keep", "K", "V", "seqlens", "idx", "w_out", "l_out", "ws"]}
INVALID, UNSUPPORTED = L.SAS_ERR_INVALID_ARG, L.SAS_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", list(NEEDED))
def test_refusals_on_the_host(name):
    for arg in NEEDED[name]:
        _expect(INVALID, lambda: _call(name, **{arg: None}))
        _expect(INVALID, lambda: _call(name, **{arg: P + 8}))
    _expect(UNSUPPORTED, lambda: _call(name, L.Shape(1, 4, 1, 96, 16, n_cap=512)))
    _expect(INVALID, lambda: _call(name, L.Shape(1, 4, 3, 64, 16, n_cap=512)))
    _expect(INVALID, lambda: _call(name, L.Shape(1, 4, 1, 64, 16, 0, 64, 8, 8)))  # paged, no table
    if name in ("append", "chunk"):
        for n in (0, -3):
            _expect(INVALID, lambda: _call(name, n_new=n))
        _expect(UNSUPPORTED, lambda: _call(name, n_new=(1 << 22) + 1))
        least = (2 if name == "append" else 8) * 64
        for stride in (least - 8, least + 4, 0, -least, 1 << 38):
            _expect(INVALID, lambda: _call(name, stride=stride))
    else:
        for over in ([dict(sinks=-1)] if name == "window" else [dict(sinks=-1), dict(recent=-1), dict(keep_max=0)]):
            _expect(INVALID, lambda: _call(name, **over))
    if name == "chunk":
        _expect(INVALID, lambda: _call(name, sinks=-1))
        _expect(UNSUPPORTED, lambda: _call(name, L.Shape(1, 129, 1, 64, 16, n_cap=512), stride=129 * 64))
    if name in ("chunk", "window"):
        _expect(UNSUPPORTED, lambda: _call(name, L.Shape(40, 512, 512, 64, 16, n_cap=131072), stride=512 * 64))  # 2^31 rows
    if name == "window":  # the list of pages
        _expect(UNSUPPORTED, lambda: _call(name, L.Shape(1, 1 << 24, 1, 64, 16, n_cap=262144)))
    need = {"append": 256, "chunk": L.sas_chunk_workspace_bytes(SHAPE, 9), "window": L.sas_window_workspace_bytes(SHAPE, True),
            "evict": L.sas_evict_workspace_bytes(SHAPE, 4)}[name]
    assert need > 0
    _expect(INVALID, lambda: _call(name, ws_bytes=need - 1))


def test_workspace_sizes():
    assert L.sas_chunk_workspace_bytes(SHAPE, 0) == 0 and L.sas_evict_workspace_bytes(SHAPE, 0) == 0
    assert L.sas_chunk_workspace_bytes(L.Shape(1, 129, 1, 64, 16, n_cap=512), 4) == 0
    assert L.sas_window_workspace_bytes(SHAPE, True) > L.sas_window_workspace_bytes(SHAPE, False) > 0
    for shape in (SHAPE, L.Shape(1, 32, 8, 128, 32, n_cap=65536), L.Shape(300, 16, 1, 64, 16, 0, 64, 64, 4000)):
        last = 0
        for n in (1, 2, 7, 64, 65, 200, 4000, 16000, 17000, 40000, 1 << 20, 1 << 22):
            size = L.sas_chunk_workspace_bytes(shape, n)
            assert size >= last  # a session for many new tokens serves calls with few
            last = size


def test_session_refuses_layouts():
    from token_level_sparse_head_b200.session import _tokens

    x = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    assert _tokens(x, 4, 64, "x") == (5, 256)
    assert _tokens(torch.zeros(5, 9, 64, dtype=torch.bfloat16)[:, 2:6], 4, 64, "x") == (5, 576)
    assert _tokens(x[:1], 4, 64, "x") == (1, 256)
    for bad in (x.float(), x[0], x.transpose(0, 1), torch.zeros(5, 8, 64, dtype=torch.bfloat16)[:, ::2],
                torch.zeros(5, 4, 128, dtype=torch.bfloat16)[:, :, ::2], x[:, :3]):
        with pytest.raises(ValueError):
            _tokens(bad, 4, 64, "x")


# ------------------------------------------------------------------------------------ values the device sees
@pytest.mark.gpu
def test_tensors_of_another_device_are_refused(cuda_lib):
    p = make_problem(B=1, Hq=4, Hkv=2, d=64, r=16, seqlens=[100], k=1, paged=False, seed=4).to("cuda")
    s = lib_and_session(p, chunk=4, window=True, evict=True)
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    start = starts_of([4]).cuda()
    with pytest.raises(ValueError):
        s.chunk(q, start.cpu(), p.K, p.V, None, p.seqlens)
    with pytest.raises(ValueError):
        s.window(p.q, p.K.cpu(), p.V, None, p.seqlens, 0)
    with pytest.raises(ValueError):
        s.append_chunk(q[:, :2], q[:, :2], start, p.M, p.K, p.V, None, None, p.seqlens.cpu())
    with pytest.raises(ValueError):
        s.evict(torch.zeros(1, 2, p.cap), torch.ones(1, dtype=torch.int32, device="cuda"), 0, 0, p.K, p.V, None, None, None, p.seqlens)
    with pytest.raises(ValueError):
        s.chunk(torch.zeros(5, 4, 64, dtype=torch.bfloat16, device="cuda"), start, p.K, p.V, None, p.seqlens)


@pytest.mark.gpu
def test_bad_chunks_are_reported_and_skipped(cuda_lib):
    p = make_problem(B=3, Hq=4, Hkv=2, d=64, r=16, seqlens=[300, 100, 200], k=1, paged=True, seed=4)
    c = p.to("cuda")
    s = lib_and_session(c, chunk=64)
    n_new = 40
    q = torch.randn(n_new, 4, 64).to(torch.bfloat16)
    kv = torch.randn(n_new, 2, 64).to(torch.bfloat16).cuda()
    new = [10, 10, 20]
    good = starts_of(new).tolist()
    kp = torch.zeros(*p.K.shape[:3], 16, dtype=torch.bfloat16, device="cuda")

    def run(start, lens=(300, 100, 200)):
        out = torch.full((n_new, 4, 64), 7.0, device="cuda", dtype=torch.bfloat16)
        lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st = torch.tensor(start, dtype=torch.int32, device="cuda")
        s.chunk(q.cuda(), st, c.K, c.V, c.page_table, lens, out=out)
        a = s.check()
        K, V = c.K.clone(), c.V.clone()
        s.append_chunk(kv, kv, st, c.M, K, V, kp, c.page_table, lens)
        b = s.check()
        return out, a, b, K

    ref, a, b, K_ref = run(good)
    assert a[0] == 0 and b[0] == 0
    check_chunk(p, q, ref, None, np.full(ref.shape, 7.0), new, 0, 0)
    untouched = torch.full_like(ref, 7.0)
    # the middle sequence out of order: only the first one is certain to be what it was
    out, a, b, _ = run([0, 10, 5, 40])
    assert a[1] == 6 and torch.equal(out[:10], ref[:10])
    # the last one past the end of the arrays
    out, a, b, _ = run([0, 10, 20, 41])
    assert a[1:] == (6, 2) and torch.equal(out[:20], ref[:20]) and torch.equal(out[20:], untouched[20:])
    assert b[1:] == (6, 2)
    # negative
    out, a, b, _ = run([-1, 10, 20, 40])
    assert a[1:] == (6, 0) and torch.equal(out[10:], ref[10:]) and torch.equal(out[:10], untouched[:10])
    # more new tokens than cached ones
    out, a, b, K = run(good, (300, 9, 200))
    assert a[1:] == (6, 1) and b[1:] == (6, 1) and torch.equal(out[10:20], untouched[10:20])
    assert torch.equal(out[:10], ref[:10]) and torch.equal(out[20:], ref[20:])
    # a length outside the cache
    out, a, b, K = run(good, (300, 100, 1 << 20))
    assert a[1:] == (1, 2) and b[1:] == (1, 2) and torch.equal(out[:20], ref[:20]) and torch.equal(out[20:], untouched[20:])
    # overlapping sequences (0..40, none, 0..40 again do not fit what the host announced): reported, nothing out of bounds
    out, a, b, _ = run([0, 40, 0, 40])
    assert a[1] == 6
    # a bad page: the other sequences are what they were
    bad = c.page_table.clone()
    bad[1, 0] = p.num_pages + 3
    out = torch.full_like(ref, 7.0)
    s.chunk(q.cuda(), torch.tensor(good, dtype=torch.int32, device="cuda"), c.K, c.V, bad, c.seqlens, out=out)
    assert s.check()[1:] == (2, 1)
    assert torch.equal(out[:10], ref[:10]) and torch.equal(out[20:], ref[20:]) and torch.isfinite(out[10:20].float()).all()
    assert run(good)[1][0] == 0


@pytest.mark.gpu
def test_nothing_new(cuda_lib):
    """Rows that belong to no sequence, and no row that does: nothing is written, nothing reported."""
    p = make_problem(B=2, Hq=4, Hkv=2, d=64, r=16, seqlens=[0, 70], k=1, paged=True, seed=4).to("cuda")
    s = lib_and_session(p, chunk=3)
    q = torch.randn(3, 4, 64, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 7.0)
    K, V = p.K.clone(), p.V.clone()
    start = starts_of([0, 0]).cuda()
    s.append_chunk(q[:, :2], q[:, 2:], start, None, K, V, None, p.page_table, p.seqlens)
    s.chunk(q, start, K, V, p.page_table, p.seqlens, out=out)
    assert s.check()[0] == 0 and (out == 7).all() and torch.equal(K, p.K) and torch.equal(V, p.V)


@pytest.mark.gpu
def test_evict_bad_values_are_reported(cuda_lib):
    p = make_problem(B=2, Hq=2, Hkv=2, d=64, r=16, seqlens=[300, 200], k=1, paged=True, seed=4).to("cuda")
    s = lib_and_session(p, k_max=50, evict=True)
    w = torch.rand(2, 2, p.cap, device="cuda")

    def run(keep, lens=(300, 200), pt=p.page_table):
        K, lo = p.K.clone(), torch.zeros(2, dtype=torch.int32, device="cuda")
        s.evict(w, torch.tensor(keep, dtype=torch.int32, device="cuda"), 0, 0, K, p.V.clone(), None, None, pt,
                torch.tensor(lens, dtype=torch.int32, device="cuda"), weights_out=torch.empty_like(w), seqlens_out=lo)
        return lo.tolist(), s.check()

    assert run([50, 20]) == ([50, 20], (0, 0, 0))
    lo, e = run([51, 20])
    assert lo == [50, 20] and e[1:] == (4, 0)
    lo, e = run([50, 20], (300, -1))
    assert lo == [50, 0] and e[1:] == (1, 1)
    bad = p.page_table.clone()
    bad[0, 0] = -5
    assert run([50, 20], pt=bad)[1][1:] == (2, 0)
    assert run([50, 20]) == ([50, 20], (0, 0, 0))


# ------------------------------------------------------------------------------------ large batches and caches
def check_rows(p, q, out, lse, new, window, sinks, tokens):
    """Chosen tokens (b, t) of a chunk against the oracle, all heads."""
    G, sigma, at = p.Hq // p.Hkv, p.d ** -0.5, [0] + list(np.cumsum(new))
    for b, t in tokens:
        n = int(p.seqlens[b])
        pos = np.nonzero(C.visible(n - new[b] + t, n, window, sinks))[0]
        for h in range(p.Hkv):
            k, v = rows(p, p.K, b, h, pos), rows(p, p.V, b, h, pos)
            ro, rl, w, W, pv = errors_of(f64(q[at[b] + t, h * G:(h + 1) * G]), k, v, sigma, p.d)
            o = f64(out[at[b] + t, h * G:(h + 1) * G])
            tol = (W + (len(pos) + 64) * 2 * U + BF) * pv + BF * np.abs(ro) + 1e-30
            assert np.all(np.abs(o - ro) <= tol), (b, t, h, np.max(np.abs(o - ro) / tol))
            assert np.all(np.abs(f64(lse[at[b] + t, h * G:(h + 1) * G]) - rl) <= W[:, 0] + 2.0 ** -21 * (1 + np.abs(rl)))


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,d,lens,new,paged,window", [
    (1, 32, 8, 128, [17000], [17000], False, 0),              # more task slots than a CTA lists, several waves
    (1, 32, 8, 128, [14400], [600], True, 0),                 # several waves, lists made by the CTAs
    (1, 12, 4, 64, [60000], [1500], True, 0),                 # waves with d = 64 and groups of 3
    (2, 16, 1, 128, [9000, 70000], [1, 900], True, 3000),     # one KV head
    (1100, 2, 1, 64, None, None, True, 0),                    # more sequences than the planning threads
])
def test_chunk_large(cuda_lib, B, Hq, Hkv, d, lens, new, paged, window):
    rng = np.random.default_rng(3)
    if lens is None:
        lens = [int(x) for x in rng.integers(1, 90, B)]
        new = [int(min(n, x)) for n, x in zip(lens, rng.integers(0, 40, B))]
    p = make_problem(B=B, Hq=Hq, Hkv=Hkv, d=d, r=16, seqlens=lens, k=1, paged=paged, seed=3)
    c = p.to("cuda")
    total = sum(new) + 2
    s = lib_and_session(c, chunk=total)
    q = torch.randn(total, Hq, d, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    lse = torch.empty(total, Hq, device="cuda")
    out, _ = s.chunk(q.cuda(), starts_of(new).cuda(), c.K, c.V, c.page_table, c.seqlens, window, 4, lse=lse)
    assert s.check()[0] == 0
    if B == 1:
        tokens = [(0, t) for t in (0, 31, 32, 63, 64, 65, new[0] // 2, new[0] // 2 + 33, new[0] - 2, new[0] - 1)]
    else:
        tokens = [(b, t) for b in range(0, B, max(1, B // 60)) for t in {0, new[b] // 2, new[b] - 1} if 0 <= t < new[b]]
    check_rows(p, q, out, lse, new, window, 4, tokens)
    again, _ = s.chunk(q.cuda(), starts_of(new).cuda(), c.K, c.V, c.page_table, c.seqlens, window, 4)
    assert torch.equal(again[:-2], out[:-2])  # the same bits every time
    # a call with fewer tokens on the same session
    if B == 1:
        few = starts_of([3]).cuda()
        o3, _ = s.chunk(q[new[0] - 3:new[0]].cuda(), few, c.K, c.V, c.page_table, c.seqlens, window, 4)
        a, b = f64(o3), f64(out[new[0] - 3:new[0]])
        assert np.all(np.abs(a - b) <= 4 * BF * (np.abs(b) + np.abs(b).max()))  # two roundings of weights and results


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d,n,T,paged", [
    (32, 8, 128, 20000, 600, True),     # two waves of KV heads, lists made by the CTAs
    (16, 8, 64, 45000, 1500, False),
    (32, 8, 128, 19500, 19500, True),   # and a list made beforehand
    (24, 6, 128, 90000, 500, False),    # four waves of one or two heads
])
def test_chunk_waves(cuda_lib, Hq, Hkv, d, n, T, paged):
    p = make_problem(B=1, Hq=Hq, Hkv=Hkv, d=d, r=16, seqlens=[n], k=1, paged=paged, seed=7)
    c = p.to("cuda")
    s = lib_and_session(c, chunk=T)
    q = torch.randn(T, Hq, d, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    lse = torch.empty(T, Hq, device="cuda")
    out, _ = s.chunk(q.cuda(), starts_of([T]).cuda(), c.K, c.V, c.page_table, c.seqlens, lse=lse)
    assert s.check()[0] == 0
    check_rows(p, q, out, lse, [T], 0, 0, [(0, t) for t in (0, 33, 64, T // 2, T - 65, T - 1)])


@pytest.mark.gpu
def test_offsets_past_32_bits(cuda_lib):
    """A cache of 2.4e9 elements per array: the last head lies behind every 32-bit element offset."""
    H, n, d, T, W = 72, 262144, 128, 40, 300
    K = torch.zeros(1, H, n, d, dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    assert K.numel() > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    heads = [0, 35, 71]
    for h in heads:
        K[0, h, -2000:] = torch.randn(2000, d, generator=g, device="cuda").to(torch.bfloat16)
        V[0, h, -2000:] = torch.randn(2000, d, generator=g, device="cuda").to(torch.bfloat16)
    from token_level_sparse_head_b200 import DecodeSession

    s = DecodeSession(L.Shape(1, H, H, d, 16, n_cap=n), 900, dense=False, chunk=T, window=True, weights=True, evict=True)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    new = torch.randn(T, 3 * H, d, generator=g, device="cuda").to(torch.bfloat16)
    q, kn, vn = new[:, :H], new[:, H:2 * H], new[:, 2 * H:]
    start = starts_of([T]).cuda()
    s.append_chunk(kn, vn, start, None, K, V, None, None, lens)
    for h in heads:
        assert torch.equal(K[0, h, -T:], kn[:, h]) and torch.equal(V[0, h, -T:], vn[:, h])
    out, _ = s.chunk(q, start, K, V, None, lens, W, 0)
    acc = torch.zeros(1, H, n, device="cuda")
    one, _ = s.window(q[-1:].contiguous(), K, V, None, lens, W, 0, weights=acc)
    for h in heads:
        z = (q[-1, h].double() @ K[0, h, -W:].double().T) * d ** -0.5
        w = torch.softmax(z, -1)
        ref = w @ V[0, h, -W:].double()
        size = (w @ V[0, h, -W:].double().abs())
        assert ((one[0, h].double() - ref).abs() <= 1e-4 * size).all()
        assert ((out[-1, h].double() - ref).abs() <= BF * 1.1 * (size + ref.abs())).all()
        assert ((acc[0, h, -W:].double() - w).abs() <= 1e-4 * w).all() and acc[0, h, :-W].abs().max() == 0
    before = {h: (K[0, h, -W:].clone(), V[0, h, -W:].clone()) for h in heads}
    s.evict(acc, torch.tensor([W], dtype=torch.int32, device="cuda"), 0, 0, K, V, None, None, None, lens)
    assert lens.tolist() == [W] and s.check()[0] == 0
    for h in heads:
        assert torch.equal(K[0, h, :W], before[h][0]) and torch.equal(V[0, h, :W], before[h][1])


# ------------------------------------------------------------------------------------ streams and graphs
@pytest.mark.gpu
def test_graphs_and_streams(cuda_lib):
    """Two captured graphs on one workspace, replayed in turn, and two sessions on two streams at once."""
    lens, new = [900, 333], [70, 40]
    p = make_problem(B=2, Hq=8, Hkv=2, d=128, r=16, seqlens=lens, k=1, paged=True, seed=5).to("cuda")
    total = sum(new)
    q = torch.randn(total, 8, 128, device="cuda").to(torch.bfloat16)
    start = starts_of(new).cuda()
    a, b = lib_and_session(p, k_max=200, chunk=total, window=True, weights=True, evict=True), None
    keep = torch.tensor([200, 100], dtype=torch.int32, device="cuda")
    K, V, lo = p.K.clone(), p.V.clone(), torch.zeros(2, dtype=torch.int32, device="cuda")
    acc, acc_out = torch.zeros(2, 2, p.cap, device="cuda"), torch.zeros(2, 2, p.cap, device="cuda")
    out, one = torch.zeros(total, 8, 128, device="cuda", dtype=torch.bfloat16), torch.zeros(2, 8, 128, device="cuda")

    def first():
        a.append_chunk(q[:, :2], q[:, 2:4], start, None, K, V, None, p.page_table, p.seqlens)
        a.chunk(q, start, K, V, p.page_table, p.seqlens, 200, 4, out=out)

    def second():
        acc.zero_()
        a.window(p.q, K, V, p.page_table, p.seqlens, 0, weights=acc, out=one)
        a.evict(acc, keep, 4, 16, K, V, None, None, p.page_table, p.seqlens, weights_out=acc_out, seqlens_out=lo)

    def start_over():
        K.copy_(p.K), V.copy_(p.V), out.zero_(), one.zero_(), acc_out.zero_(), lo.zero_()

    start_over(), first(), second()
    want = [t.clone() for t in (out, one, K, V, acc_out, lo)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for f in (first, second):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                f()
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        start_over()
        graphs[0].replay()
        graphs[1].replay()
        for x, y in zip((out, one, K, V, acc_out, lo), want):
            assert torch.equal(x, y)
    # another session on another stream at the same time
    b = lib_and_session(p, k_max=200, chunk=total, window=True)
    K2, V2 = want[2].clone(), want[3].clone()
    out2 = torch.zeros_like(out)
    refs = []
    b.chunk(q, start, K2, V2, p.page_table, p.seqlens, out=out2)
    refs.append(out2.clone())
    start_over()
    torch.cuda.synchronize()
    for _ in range(10):
        first()
        with torch.cuda.stream(side):
            b.chunk(q, start, K2, V2, p.page_table, p.seqlens, out=out2)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(out2, refs[0])
    assert a.check()[0] == 0 and b.check()[0] == 0


# ------------------------------------------------------------------------------------ together
@pytest.mark.gpu
@pytest.mark.parametrize("paged,fp8", [(True, False), (False, True)])
def test_prompt_decode_evict_and_drafts(cuda_lib, paged, fp8):
    """A prompt into an empty cache and through the attention, decoded tokens with accumulated weights, an
    eviction, drafted tokens over what is left, and a sparse step on the same workspace."""
    B, Hq, Hkv, d, r = 2, 8, 2, 128, 16
    prompt, steps, drafts, keep, sinks, recent = [700, 301], 3, 5, [200, 150], 4, 32
    top = [n + steps for n in prompt]
    p = make_problem(B=B, Hq=Hq, Hkv=Hkv, d=d, r=r, seqlens=top, k=64, paged=paged, seed=11, kproj_fp8=fp8)
    pt = None if p.page_table is None else p.page_table.numpy()
    c = p.to("cuda")
    c.K.fill_(float("nan")), c.V.fill_(float("nan"))
    K, V = f64(c.K), f64(c.V)
    s = lib_and_session(c, k_max=256, chunk=1100, weights=True, evict=True)
    kp = torch.zeros(*p.K.shape[:3], r, dtype=torch.float8_e4m3fn if fp8 else torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(12)
    acc = torch.zeros(B, Hkv, p.cap, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def put(new, counts):
        nonlocal K, V
        lens.add_(torch.tensor(counts, dtype=torch.int32, device="cuda"))
        start = starts_of(counts)
        x = new.cuda()
        k, v = x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        s.append_chunk(k, v, start.cuda(), c.M, c.K, c.V, kp, c.page_table, lens)
        K, V = C.append_chunk(K, V, f64(k), f64(v), start.numpy(), lens.tolist(), pt)
        return x[:, :Hq], start.cuda()

    def now(q=None):
        view = make_problem(B=B, Hq=Hq, Hkv=Hkv, d=d, r=r, seqlens=lens.tolist(), k=1, paged=False, seed=1)
        view.K, view.V, view.page_table, view.q = c.K.cpu(), c.V.cpu(), p.page_table, q
        return view

    rows_of = lambda n: torch.randn(n, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16)  # noqa: E731
    q, start = put(rows_of(sum(prompt)), prompt)
    assert np.array_equal(f64(c.K), K, equal_nan=True) and np.array_equal(f64(c.V), V, equal_nan=True)
    out, _ = s.chunk(q, start, c.K, c.V, c.page_table, lens)
    check_chunk(now(), q, out, None, np.zeros((sum(prompt), Hq, d)), prompt, 0, 0)
    for _ in range(steps):
        q, start = put(rows_of(B), [1] * B)
        was = acc.clone()
        one, lse = s.window(q.contiguous(), c.K, c.V, c.page_table, lens, 0, weights=acc, lse=torch.empty(B, Hq, device="cuda"))
        check_window(now(q.cpu()), one, lse, acc, was.cpu(), 0, 0)
    kept = [[C.evict_positions(acc[b, h].cpu().numpy(), top[b], keep[b], sinks, recent) for h in range(Hkv)] for b in range(B)]
    s.evict(acc, torch.tensor(keep, dtype=torch.int32, device="cuda"), sinks, recent, c.K, c.V, kp, None, c.page_table, lens)
    assert lens.tolist() == keep
    for b in range(B):
        for h in range(Hkv):
            i1, i3 = C.slot(pt, b, kept[b][h])
            o1, o3 = C.slot(pt, b, np.arange(keep[b]))
            for x in (K, V):
                x[o1, h, o3] = x[i1, h, i3].copy()
    assert np.array_equal(f64(c.K), K, equal_nan=True) and np.array_equal(f64(c.V), V, equal_nan=True)
    q, start = put(rows_of(B * drafts), [drafts] * B)
    out, _ = s.chunk(q, start, c.K, c.V, c.page_table, lens, 100, 4)
    check_chunk(now(), q, out, None, np.zeros((B * drafts, Hq, d)), [drafts] * B, 100, 4)
    # the projected rows went along: they are the build's over the rows as they lie now
    want = kp.clone()
    cuda_lib.sas_build_proj_cache(s.shape, c.K, c.M, want, c.page_table, lens)
    assert torch.equal(want.view(torch.uint8), kp.view(torch.uint8))
    # a sparse step over every row is the dense one
    q1 = q[[drafts - 1, 2 * drafts - 1]].contiguous()
    k_all = torch.full((B,), 256, dtype=torch.int32, device="cuda")
    sparse, _ = s.decode(q1, c.M, kp, c.K, c.V, c.page_table, lens, k_all, out=torch.empty(B, Hq, d, device="cuda"))
    dense, _ = s.window(q1, c.K, c.V, c.page_table, lens, 0, out=torch.empty(B, Hq, d, device="cuda"))
    assert (sparse - dense).abs().max() < 1e-5 and s.check()[0] == 0
