"""What a call may read before the kernel launched ahead of it has completed.

Every kernel is launched so that its set-up may overlap the end of the kernel before it; only its
wait makes that kernel's writes visible.  The first kernel of a call follows another call's kernel or
the caller's own, which may have written any of the call's inputs (an eviction writes the lengths),
so it waits before it reads one.
"""
import os
import re

import pytest
import torch

from synth import make_problem
from tests.test_cache_ops import lib_and_session

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "token_level_sparse_head_b200", "csrc")
# the kernels that can be the first of a call, and the wait that such a launch reaches
FIRST = [("score.cu", "score_kernel"), ("attend.cu", "attend_kernel"), ("select.cu", "select_topk_kernel"),
         ("proj.cu", "build_kernel"), ("proj.cu", "append_kernel"), ("gather.cu", "gather_kernel"), ("append.cu", "token_kernel"),
         ("append.cu", "tile_kernel"), ("chunk.cu", "plan_kernel"), ("chunk.cu", "chunk_kernel"), ("window.cu", "window_kernel"),
         ("evict.cu", "evict_keys_kernel")]
READS = re.compile(r"p\.(seqlens|kvec|keep|q|idx|q_start|page_table|weights|log_g|K|V|kproj|K_new|V_new|M|keys|hist)\b(?!\w)|seq_info<|seq_len\(")


@pytest.mark.parametrize("file,kernel", FIRST)
def test_first_kernels_wait_before_they_read(file, kernel):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
    at = re.search(r"__global__[^;{]*?\b" + kernel + r"\([^)]*\)\s*\{", text)
    assert at, kernel
    body = text[at.end():]
    before = body[:body.index("pdl_wait()")]
    found = READS.search(before)
    assert found is None, f"{kernel} reads {found.group(0)} before its wait"


@pytest.mark.gpu
@pytest.mark.parametrize("paged,B", [(True, 4), (False, 1)])
def test_lengths_written_right_before_a_call(cuda_lib, paged, B):
    """An eviction in place, then a step, a dense decode, a selection and an attention with nothing in
    between, replayed; the results are those of the same calls one at a time."""
    lens = [9000, 700, 4097, 65][:B]
    keep = [1500, 600, 64, 3][:B]
    p = make_problem(B=B, Hq=8, Hkv=2, d=128, r=16, seqlens=lens, k=[300, 100, 64, 2][:B], k_max=2000, paged=paged, seed=31).to("cuda")
    s = lib_and_session(p, k_max=2000, dense=True, evict=True)
    kp0 = torch.zeros(*p.K.shape[:3], 16, dtype=torch.bfloat16, device="cuda")
    cuda_lib.sas_build_proj_cache(s.shape, p.K, p.M, kp0, p.page_table, p.seqlens)
    K, V, kp, n = p.K.clone(), p.V.clone(), kp0.clone(), p.seqlens.clone()
    w0 = torch.rand(B, 2, p.cap, device="cuda")
    w = w0.clone()
    keep_d = torch.tensor(keep, dtype=torch.int32, device="cuda")
    kept = torch.empty(B, 2, 2000, dtype=torch.int32, device="cuda")
    out = {name: torch.zeros(B, 8, 128, device="cuda") for name in ("step", "dense", "attend")}
    idx = {name: torch.zeros(B, 2, 2000, dtype=torch.int32, device="cuda") for name in ("step", "select")}
    calls = {
        "step": lambda: s.decode(p.q, p.M, kp, K, V, p.page_table, n, p.k, out=out["step"], idx=idx["step"]),
        "dense": lambda: s.dense(p.q, K, V, p.page_table, n, out=out["dense"]),
        "select": lambda: s.select(p.q, p.M, kp, p.page_table, n, p.k, idx=idx["select"]),
        "attend": lambda: s.attend(p.q, K, V, p.page_table, n, idx["select"], p.k, out=out["attend"]),
    }

    def run(name, wait):
        K.copy_(p.K), V.copy_(p.V), kp.copy_(kp0), w.copy_(w0), n.copy_(p.seqlens)
        s.evict(w, keep_d, 4, 16, K, V, kp, None, p.page_table, n, idx=kept)
        wait()
        calls[name]()

    for name in ("step", "dense", "select", "attend"):
        result = [out[name]] if name in out else []
        result += [idx[name]] if name in idx else []
        run(name, torch.cuda.synchronize)
        want = [x.clone() for x in result]
        assert n.tolist() == [min(a, b) for a, b in zip(lens, keep)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(name, lambda: None)
        for i in range(40):
            for x in result:
                x.zero_()
            g.replay() if i % 2 else run(name, lambda: None)
            for x, y in zip(result, want):
                assert torch.equal(x, y), (name, i)
    assert s.check()[0] == 0
