"""DecodeSession: owns the workspace for one problem shape and forwards to the C ABI.

PyTorch provides the device memory (workspace, outputs) and the stream; the library does
all the work.
"""
from __future__ import annotations

import torch

from . import lib


def _tokens(x, heads: int, d: int, name: str):
    """Tokens and token stride of a bf16 [n][heads][d] tensor whose heads are dense."""
    size, step = tuple(x.shape), x.stride()
    if x.dtype != torch.bfloat16 or size[1:] != (heads, d) or len(size) != 3:
        raise ValueError(f"{name} must be bf16 [tokens][{heads}][{d}], got {x.dtype} {size}")
    if step[2] != 1 or (heads > 1 and step[1] != d):
        raise ValueError(f"{name}: the heads of a token must lie one after another")
    return size[0], step[0] if size[0] > 1 else heads * d


def _other_layout(x, dtype, shape) -> bool:
    """x is neither dense [shape] of dtype nor more of the same along the first axis."""
    size = x.shape
    return x.dtype is not dtype or not x.is_contiguous() or len(size) != len(shape) or size[1:] != shape[1:] or size[0] < shape[0]


class _Sizes:
    """A session's shape as the calls take it: the C structure is made once (0.8 us), the scale's address is the
    shape's of now."""

    def __init__(self, shape: lib.Shape):
        self.shape, self._c = shape, shape.c()

    def c(self):
        self._c.kproj_scale = lib._p(self.shape.kproj_scale)
        return self._c


class DecodeSession:
    """Workspace + output buffers for repeated decode steps of one shape and budget bound.

    chunk: the most new tokens a call of chunk() takes (0: chunk() is not used).
    window, weights: window() is used, and whether with accumulated weights.
    evict: evict() is used, with budgets of at most k_max rows.
    """

    def __init__(self, shape: lib.Shape, k_max: int, device="cuda", dense: bool = True, chunk: int = 0,
                 window: bool = False, weights: bool = False, evict: bool = False):
        self.shape = shape
        self._sizes = _Sizes(shape)
        self.k_max = int(k_max)
        self.chunk_max = int(chunk)
        # (name, type, extents) of what the calls around the step take; there may be more along the first axis
        s, i32, f32, bf16 = shape, torch.int32, torch.float32, torch.bfloat16
        self._rows = (s.num_pages, s.Hkv, s.page_size) if s.page_size else (s.B, s.Hkv, s.n_cap)
        positions, heads = (s.B, s.Hkv, s.cap), (s.B, s.Hq, s.d)
        self._starts, self._m = ("q_start", i32, (s.B + 1,)), ("M", f32, (s.Hkv, s.r, s.d))
        self._cache = (("K", bf16, (*self._rows, s.d)), ("V", bf16, (*self._rows, s.d)), ("seqlens", i32, (s.B,)),
                       ("page_table", i32, (s.B, s.max_pages)) if s.page_size else None)
        self._window = (*self._cache, ("q", bf16, heads), ("out", f32, heads), ("lse", f32, (s.B, s.Hq)), ("weights", f32, positions))
        self._evict = (*self._cache, ("weights", f32, positions), ("keep", i32, (s.B,)), ("log_g", f32, positions), ("idx", i32, (s.B, s.Hkv, self.k_max)),
                       ("weights_out", f32, positions), ("seqlens_out", i32, (s.B,)))
        sizes = [lib.sas_decode_workspace_bytes(shape, self.k_max)]
        if dense:
            sizes.append(lib.sas_dense_workspace_bytes(shape))
        if chunk:
            sizes.append(lib.sas_chunk_workspace_bytes(shape, self.chunk_max))
        if window or weights:
            sizes.append(lib.sas_window_workspace_bytes(shape, weights))
        if evict:
            sizes.append(lib.sas_evict_workspace_bytes(shape, self.k_max))
        if min(sizes) == 0:
            raise ValueError("invalid shape for libsas")
        nbytes = max(sizes)
        self.ws_bytes = nbytes
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.device = self.workspace.device
        with torch.cuda.device(self.device):
            lib.sas_workspace_init(self.workspace, nbytes)
        self.out = torch.empty(shape.B, shape.Hq, shape.d, dtype=torch.float32, device=device)
        self.idx = torch.empty(shape.B, shape.Hkv, self.k_max, dtype=torch.int32, device=device)

    def decode(self, q, M, Kproj, K, V, page_table, seqlens, k, lam=0.0, log_g=None, out=None, idx=None):
        out = self.out if out is None else out
        idx = self.idx if idx is None else idx
        self._launch(lib.sas_decode_step, q, M, Kproj, K, V, page_table, seqlens, k, self.k_max, lam, log_g, out, idx)
        return out, idx

    def dense(self, q, K, V, page_table, seqlens, out=None):
        out = self.out if out is None else out
        self._launch(lib.sas_dense_decode, q, K, V, page_table, seqlens, out)
        return out

    def select(self, q, M, Kproj, page_table, seqlens, k, lam=0.0, log_g=None, idx=None, scores=None):
        idx = self.idx if idx is None else idx
        self._launch(lib.sas_select_topk, q, M, Kproj, page_table, seqlens, k, self.k_max, lam, log_g, idx, scores)
        return idx

    def attend(self, q, K, V, page_table, seqlens, idx, k, lam=0.0, log_g=None, out=None):
        out = self.out if out is None else out
        self._launch(lib.sas_sparse_attention, q, K, V, page_table, seqlens, idx, k, self.k_max, lam, log_g, out)
        return out

    def _launch(self, call, *args):
        """A call on the session's device and that device's current stream."""
        index = self.device.index
        if torch.cuda.current_device() == index:
            call(self._sizes, *args, self.workspace, self.ws_bytes, lib._raw_stream(index))
        else:
            with torch.cuda.device(index):
                call(self._sizes, *args, self.workspace, self.ws_bytes, lib._raw_stream(index))

    def _run(self, call, tensors, specs, *args):
        """A call whose tensors all lie on the session's device and, where there is a spec, have its layout: the
        library takes addresses, and would read or write another as if it had."""
        index = self.device.index
        for x, spec in zip(tensors, specs):
            if x is None:
                continue
            if x.get_device() != index:
                raise ValueError(f"a tensor lies on {x.device}, the session on {self.device}")
            if spec is None:
                continue
            name, dtype, shape = spec
            if (x.shape != shape or x.dtype is not dtype or not x.is_contiguous()) and _other_layout(x, dtype, shape):
                raise ValueError(f"{name} must be contiguous {dtype} {list(shape)}, got {x.dtype} {list(x.shape)} with strides {x.stride()}")
        self._launch(call, *args)

    def _projected(self, Kproj):
        """Spec of projected rows, as values or as their bytes."""
        if Kproj is None:
            return None
        row = self.shape.r * (1 if self.shape.kproj_dtype == lib.SAS_KPROJ_FP8_E4M3 else 2)
        return ("Kproj", Kproj.dtype, (*self._rows, row // Kproj.element_size()))

    def append_chunk(self, K_new, V_new, q_start, M, K, V, Kproj, page_table, seqlens):
        """K_new, V_new [n_new][Hkv][d], tokens at any stride; Kproj (and M) may be None."""
        n_new, stride = _tokens(K_new, self.shape.Hkv, self.shape.d, "K_new")
        if _tokens(V_new, self.shape.Hkv, self.shape.d, "V_new") != (n_new, stride):
            raise ValueError("K_new and V_new differ in tokens or stride")
        self._run(lib.sas_append_chunk, (K, V, seqlens, page_table, q_start, M, Kproj, K_new, V_new),
                  (*self._cache, self._starts, self._m, self._projected(Kproj), None, None),
                  K_new, V_new, stride, q_start, n_new, M, K, V, Kproj, page_table, seqlens)

    def chunk(self, q, q_start, K, V, page_table, seqlens, window=0, sinks=0, out=None, lse=None):
        """q [n_new][Hq][d], tokens at any stride.  Returns out (bf16) and lse (None unless given)."""
        Hq, d = self.shape.Hq, self.shape.d
        n_new, stride = _tokens(q, Hq, d, "q")
        if n_new > self.chunk_max:
            raise ValueError(f"{n_new} new tokens, more than the session's {self.chunk_max}")
        if out is None:
            out = torch.empty(n_new, Hq, d, dtype=torch.bfloat16, device=q.device)
        self._run(lib.sas_chunk_attention, (K, V, seqlens, page_table, q_start, out, lse, q),
                  (*self._cache, self._starts, ("out", torch.bfloat16, (n_new, Hq, d)), ("lse", torch.float32, (n_new, Hq)), None),
                  q, stride, q_start, n_new, K, V, page_table, seqlens, window, sinks, out, lse)
        return out, lse

    def window(self, q, K, V, page_table, seqlens, window, sinks=0, weights=None, out=None, lse=None):
        """The newest token of every sequence, q dense.  Adds the softmax weights to `weights` unless None."""
        out = self.out if out is None else out
        self._run(lib.sas_window_decode, (K, V, seqlens, page_table, q, out, lse, weights), self._window,
                  q, K, V, page_table, seqlens, window, sinks, out, lse, weights)
        return out, lse

    def evict(self, weights, keep, sinks, recent, K, V, Kproj, log_g, page_table, seqlens, idx=None, weights_out=None,
              seqlens_out=None):
        """In place by default: weights and seqlens are updated where they are."""
        idx = self.idx if idx is None else idx
        weights_out = weights if weights_out is None else weights_out
        seqlens_out = seqlens if seqlens_out is None else seqlens_out
        self._run(lib.sas_evict, (K, V, seqlens, page_table, weights, keep, log_g, idx, weights_out, seqlens_out, Kproj),
                  (*self._evict, self._projected(Kproj)),
                  weights, keep, self.k_max, sinks, recent, K, V, Kproj, log_g, page_table, seqlens, idx, weights_out,
                  seqlens_out)
        return idx

    def check(self):
        """(status, code, where) of the device-side checks since the last check (synchronises)."""
        with torch.cuda.device(self.device):
            return lib.sas_check_workspace(self.workspace, self.ws_bytes)
