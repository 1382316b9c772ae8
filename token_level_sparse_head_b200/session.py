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


class DecodeSession:
    """Workspace + output buffers for repeated decode steps of one shape and budget bound.

    chunk: the most new tokens a call of chunk() takes (0: chunk() is not used).
    window, weights: window() is used, and whether with accumulated weights.
    evict: evict() is used, with budgets of at most k_max rows.
    """

    def __init__(self, shape: lib.Shape, k_max: int, device="cuda", dense: bool = True, chunk: int = 0,
                 window: bool = False, weights: bool = False, evict: bool = False):
        self.shape = shape
        self.k_max = int(k_max)
        self.chunk_max = int(chunk)
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
        lib.sas_workspace_init(self.workspace, nbytes)
        self.device = self.workspace.device
        self.out = torch.empty(shape.B, shape.Hq, shape.d, dtype=torch.float32, device=device)
        self.idx = torch.empty(shape.B, shape.Hkv, self.k_max, dtype=torch.int32, device=device)

    def decode(self, q, M, Kproj, K, V, page_table, seqlens, k, lam=0.0, log_g=None, out=None, idx=None):
        out = self.out if out is None else out
        idx = self.idx if idx is None else idx
        lib.sas_decode_step(self.shape, q, M, Kproj, K, V, page_table, seqlens, k, self.k_max, lam, log_g,
                            out, idx, self.workspace, self.ws_bytes)
        return out, idx

    def dense(self, q, K, V, page_table, seqlens, out=None):
        out = self.out if out is None else out
        lib.sas_dense_decode(self.shape, q, K, V, page_table, seqlens, out, self.workspace, self.ws_bytes)
        return out

    def select(self, q, M, Kproj, page_table, seqlens, k, lam=0.0, log_g=None, idx=None, scores=None):
        idx = self.idx if idx is None else idx
        lib.sas_select_topk(self.shape, q, M, Kproj, page_table, seqlens, k, self.k_max, lam, log_g, idx,
                            scores, self.workspace, self.ws_bytes)
        return idx

    def attend(self, q, K, V, page_table, seqlens, idx, k, lam=0.0, log_g=None, out=None):
        out = self.out if out is None else out
        lib.sas_sparse_attention(self.shape, q, K, V, page_table, seqlens, idx, k, self.k_max, lam, log_g,
                                 out, self.workspace, self.ws_bytes)
        return out

    def _run(self, call, tensors, *args):
        """A call on the session's device and that device's current stream; every tensor lies there."""
        index = self.device.index
        for t in tensors:
            if t is not None and t.get_device() != index:
                raise ValueError(f"a tensor lies on {t.device}, the session on {self.device}")
        if torch.cuda.current_device() == index:
            call(self.shape, *args, self.workspace, self.ws_bytes, lib._raw_stream(index))
        else:
            with torch.cuda.device(index):
                call(self.shape, *args, self.workspace, self.ws_bytes, lib._raw_stream(index))

    def append_chunk(self, K_new, V_new, q_start, M, K, V, Kproj, page_table, seqlens):
        """K_new, V_new [n_new][Hkv][d], tokens at any stride; Kproj (and M) may be None."""
        n_new, stride = _tokens(K_new, self.shape.Hkv, self.shape.d, "K_new")
        if _tokens(V_new, self.shape.Hkv, self.shape.d, "V_new") != (n_new, stride):
            raise ValueError("K_new and V_new differ in tokens or stride")
        self._run(lib.sas_append_chunk, (K_new, V_new, q_start, M, K, V, Kproj, page_table, seqlens), K_new, V_new, stride,
                  q_start, n_new, M, K, V, Kproj, page_table, seqlens)

    def chunk(self, q, q_start, K, V, page_table, seqlens, window=0, sinks=0, out=None, lse=None):
        """q [n_new][Hq][d], tokens at any stride.  Returns out (bf16) and lse (None unless given)."""
        n_new, stride = _tokens(q, self.shape.Hq, self.shape.d, "q")
        if n_new > self.chunk_max:
            raise ValueError(f"{n_new} new tokens, more than the session's {self.chunk_max}")
        if out is None:
            out = torch.empty(n_new, self.shape.Hq, self.shape.d, dtype=torch.bfloat16, device=q.device)
        self._run(lib.sas_chunk_attention, (q, q_start, K, V, page_table, seqlens, out, lse), q, stride, q_start, n_new, K, V,
                  page_table, seqlens, window, sinks, out, lse)
        return out, lse

    def window(self, q, K, V, page_table, seqlens, window, sinks=0, weights=None, out=None, lse=None):
        """The newest token of every sequence.  Adds the softmax weights to `weights` unless None."""
        out = self.out if out is None else out
        self._run(lib.sas_window_decode, (q, K, V, page_table, seqlens, weights, out, lse), q, K, V, page_table, seqlens,
                  window, sinks, out, lse, weights)
        return out, lse

    def evict(self, weights, keep, sinks, recent, K, V, Kproj, log_g, page_table, seqlens, idx=None, weights_out=None,
              seqlens_out=None):
        """In place by default: weights and seqlens are updated where they are."""
        idx = self.idx if idx is None else idx
        weights_out = weights if weights_out is None else weights_out
        seqlens_out = seqlens if seqlens_out is None else seqlens_out
        self._run(lib.sas_evict, (weights, keep, K, V, Kproj, log_g, page_table, seqlens, idx, weights_out, seqlens_out),
                  weights, keep, self.k_max, sinks, recent, K, V, Kproj, log_g, page_table, seqlens, idx, weights_out,
                  seqlens_out)
        return idx

    def check(self):
        """(status, code, where) of the device-side checks since the last check (synchronises)."""
        return lib.sas_check_workspace(self.workspace, self.ws_bytes)
