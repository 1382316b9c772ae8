"""DecodeSession refuses tensors whose type, extents or strides are not what the library reads, and works
on its own device whatever the current one is.

The library takes addresses: a tensor of another layout would be read, or written, as if it had the
right one.  On the CPU, with the library's calls recorded instead of made.
"""
import contextlib
import types

import pytest
import torch

from token_level_sparse_head_b200 import DecodeSession, Shape, lib, session

BF, F, I = torch.bfloat16, torch.float32, torch.int32
CALLS = {"append_chunk": "sas_append_chunk", "chunk": "sas_chunk_attention", "window": "sas_window_decode", "evict": "sas_evict"}


@pytest.fixture
def made(monkeypatch):
    """The library calls that were made, by name."""
    calls = []
    for name in CALLS.values():
        monkeypatch.setattr(lib, name, lambda *a, name=name: calls.append(name))
    for name in ("sas_workspace_init", "sas_check_workspace"):
        monkeypatch.setattr(lib, name, lambda *a, **k: (0, 0, 0))
    monkeypatch.setattr(lib, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    return calls


def make(paged, fp8=False):
    """A session and, by call, valid arguments."""
    B, Hq, Hkv, d, r, T = 3, 8, 2, 64, 16, 9
    scale = torch.ones(Hkv)
    shape = (Shape(B, Hq, Hkv, d, r, 0, 64, 4, 11, int(fp8), scale if fp8 else None) if paged else
             Shape(B, Hq, Hkv, d, r, 256, 0, 0, 0, int(fp8), scale if fp8 else None))
    s = DecodeSession(shape, 50, device="cpu", dense=False, chunk=20, window=True, weights=True, evict=True)
    s.device = type("Device", (), {"index": -1})()
    lead = (11, Hkv, 64) if paged else (B, Hkv, 256)
    z = torch.zeros
    cache = dict(K=z(*lead, d, dtype=BF), V=z(*lead, d, dtype=BF), page_table=z(B, 4, dtype=I) if paged else None, seqlens=z(B, dtype=I))
    kp = z(*lead, r, dtype=torch.float8_e4m3fn if fp8 else BF)
    rows = dict(q_start=z(B + 1, dtype=I))
    return s, {
        "append_chunk": dict(cache, **rows, K_new=z(T, Hkv, d, dtype=BF), V_new=z(T, Hkv, d, dtype=BF), M=z(Hkv, r, d), Kproj=kp),
        "chunk": dict(cache, **rows, q=z(T, Hq, d, dtype=BF), out=z(T, Hq, d, dtype=BF), lse=z(T, Hq)),
        "window": dict(cache, q=z(B, Hq, d, dtype=BF), window=0, weights=z(B, Hkv, 256), out=z(B, Hq, d), lse=z(B, Hq)),
        "evict": dict(cache, weights=z(B, Hkv, 256), keep=z(B, dtype=I), sinks=0, recent=0, Kproj=kp, log_g=z(B, Hkv, 256),
                      idx=z(B, Hkv, 50, dtype=I), weights_out=z(B, Hkv, 256), seqlens_out=z(B, dtype=I)),
    }


def wrong(name, x):
    """Layouts that are not x's: another type, too short, rows apart, another last extent."""
    other = {BF: F, F: BF, I: torch.int64, torch.float8_e4m3fn: BF}[x.dtype]
    if name == "Kproj":
        yield x[:-1]
    else:
        yield x.to(other)
        yield x[:-1]
    wide = torch.zeros(*x.shape[:-1], 2 * x.shape[-1], dtype=x.dtype)
    yield wide[..., ::2]
    if x.dim() > 1:
        yield wide[..., :x.shape[-1]]
        yield wide
        yield x[..., :-1].contiguous()
        yield torch.cat([x, x], dim=1)
        yield x[:, :-1].contiguous()


@pytest.mark.parametrize("paged,fp8", [(False, False), (True, True)])
@pytest.mark.parametrize("call", list(CALLS))
def test_layouts_are_refused(made, call, paged, fp8):
    s, args = make(paged, fp8)
    args = args[call]
    getattr(s, call)(**args)
    assert made == [CALLS[call]]
    made.clear()
    for name, x in args.items():
        if not isinstance(x, torch.Tensor) or name in ("K_new", "V_new") or (name == "q" and call == "chunk"):
            continue  # these take token strides and have checks of their own
        for bad in wrong(name, x):
            with pytest.raises(ValueError, match=name):
                getattr(s, call)(**dict(args, **{name: bad}))
    assert made == []


@pytest.mark.parametrize("paged", [False, True])
def test_longer_arrays_and_defaults_are_taken(made, paged):
    """More along the first axis than the call needs: buffers kept for the largest batch."""
    s, args = make(paged)
    for call, kw in args.items():
        for name, x in kw.items():
            if isinstance(x, torch.Tensor) and name not in ("K_new", "V_new", "q"):
                kw = dict(kw, **{name: torch.cat([x, x])})
        getattr(s, call)(**kw)
    s.append_chunk(**dict(args["append_chunk"], M=None, Kproj=None))
    s.chunk(**dict(args["chunk"], out=None, lse=None))
    s.window(**dict(args["window"], out=None, lse=None, weights=None))
    s.evict(**dict(args["evict"], Kproj=None, log_g=None, idx=None, weights_out=None, seqlens_out=None))
    assert len(made) == 8


def test_projected_rows_as_bytes(made):
    s, args = make(False)
    kp = args["evict"]["Kproj"]
    s.evict(**dict(args["evict"], Kproj=kp.view(torch.uint8)))
    assert made == ["sas_evict"]


def test_queries_of_a_fused_projection(made):
    """The chunk takes rows at a stride; the window takes dense ones and says so."""
    s, args = make(False)
    fused = torch.zeros(9, 12, 64, dtype=BF)
    s.chunk(**dict(args["chunk"], q=fused[:, :8]))
    with pytest.raises(ValueError, match="q must be contiguous"):
        s.window(**dict(args["window"], q=fused[:3, :8]))
    assert made == ["sas_chunk_attention"]


def test_every_call_is_made_on_the_sessions_device(monkeypatch):
    """The workspace is cleared, used and read back on streams of the device that it lies on."""
    current, made = [0], []

    @contextlib.contextmanager
    def device(d):
        was, current[0] = current[0], (7 if isinstance(d, torch.device) else d)
        yield
        current[0] = was

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(lib, "_raw_stream", lambda index: 100 + index)
    for name in ("sas_workspace_init", "sas_check_workspace"):
        monkeypatch.setattr(lib, name, lambda *a, name=name: made.append((name, current[0], 100 + current[0])))
    for name in (*CALLS.values(), "sas_decode_step", "sas_dense_decode", "sas_select_topk", "sas_sparse_attention"):
        # without a stream the library takes the current device's
        monkeypatch.setattr(lib, name, lambda *a, name=name: made.append((name, current[0], a[-1] if isinstance(a[-1], int) and a[-1] >= 100 and
                                                                            a[-1] < 200 else 100 + current[0])))
    s = DecodeSession(Shape(1, 2, 1, 64, 16, 256), 4, device="cpu", chunk=2, window=True, evict=True)
    s.device = torch.device("cuda", 7)
    x = types.SimpleNamespace(get_device=lambda: 7, shape=(), dtype=None, is_contiguous=lambda: True, stride=tuple, device="cuda:7")
    monkeypatch.setattr(session, "_other_layout", lambda *a: False)
    monkeypatch.setattr(session, "_tokens", lambda *a: (2, 128))
    s._projected = lambda kp: None
    s.decode(x, x, x, x, x, None, x, x), s.dense(x, x, x, None, x), s.select(x, x, x, None, x, x), s.attend(x, x, x, None, x, x, x)
    s.append_chunk(x, x, x, x, x, x, x, None, x), s.chunk(x, x, x, x, None, x, out=x), s.window(x, x, x, None, x, 0, out=x)
    s.evict(x, x, 0, 0, x, x, x, x, None, x, idx=x)
    s.check()
    assert len(made) == 10 and {m[1:] for m in made} == {(7, 107)}, made


def test_the_scale_is_the_shapes_of_now(made, monkeypatch):
    """The C structure is made once; a scale tensor that the caller puts in later is the one that calls get."""
    s, args = make(True, fp8=True)
    seen = []
    monkeypatch.setattr(lib, "sas_append_chunk", lambda shape, *a: seen.append((shape.c().kproj_scale, shape.c().B)))
    first = s.shape.kproj_scale
    s.append_chunk(**args["append_chunk"])
    s.shape.kproj_scale = torch.full_like(first, 2.0)
    s.append_chunk(**args["append_chunk"])
    second, s.shape.kproj_scale = s.shape.kproj_scale, None
    s.append_chunk(**args["append_chunk"])  # which the library then refuses
    assert seen == [(first.data_ptr(), 3), (second.data_ptr(), 3), (None, 3)]
