"""Cases, plain forms and exact values of the cache operators: append of a chunk, attention of a
chunk, window decode with accumulated weights, and eviction.

`run` in the plain form uses elementary torch operations in 32 bits; with `own` it makes the calls
that a user makes of the library.  Shapes follow the workloads of this repository (Hq = 32,
Hkv = 8, d = 128, r = 32, 64-token pages, 8K to 128K cached tokens).
"""
import math

import torch

own = False

PAGE = 64


# ------------------------------------------------------------------------------------ cases
def _case(name, op, **kw):
    c = dict(name=name, op=op, B=1, Hq=32, Hkv=8, d=128, r=32, paged=True, fp8=False, n_lo=4096, n_hi=4096,
             t_lo=1, t_hi=1, window=0, sinks=0, weights=False, keep_div=8, recent=0, fused=False, gate=False, pad=0)
    c.update(kw)
    return c


def listed():
    return [
        # the append of a decode step: one new token per sequence into an FP8-scored paged cache
        _case("append 16 x 1", "append", B=16, n_lo=1, n_hi=8192, fp8=True),
        # a whole prompt's rows into a contiguous cache
        _case("append 8192", "append", paged=False, n_lo=32768, n_hi=32768, t_lo=8192, t_hi=8192),
        # chunks of a mixed batch, straight from the rows of a fused projection, smaller heads
        _case("append ragged fused", "append", B=16, d=64, r=16, n_lo=2048, n_hi=8192, t_lo=1, t_hi=2047, fused=True, pad=5),
        # verification of a few drafted tokens per sequence: latency and cache bandwidth
        _case("chunk 8 x 5 drafted", "chunk", B=8, n_lo=4096, n_hi=32768, t_lo=5, t_hi=5),
        # a prompt from nothing, causal, contiguous
        _case("chunk 8192 prompt", "chunk", paged=False, n_lo=8192, n_hi=8192, t_lo=8192, t_hi=8192),
        # one chunk of a long prompt over its paged cache
        _case("chunk 512 on 32K", "chunk", n_lo=32768, n_hi=32768, t_lo=512, t_hi=512, fused=True),
        # a mixed batch of chunks and single tokens with a window and sinks, d = 64
        _case("chunk ragged window", "chunk", B=16, d=64, r=16, n_lo=600, n_hi=8192, t_lo=1, t_hi=383, window=1024, sinks=4, pad=3),
        # one sequence's decode with a window: the smallest attention call
        _case("window 1024 b1", "window", paged=False, n_lo=32768, n_hi=32768, window=1024, sinks=4),
        # a batch's decode with a window, wide head groups
        _case("window 4096 b16", "window", B=16, Hq=64, n_lo=8192, n_hi=131072, window=4096, sinks=4),
        # decode over whole caches, its weights accumulated for a later eviction
        _case("weights b4 64K", "window", B=4, paged=False, n_lo=65536, n_hi=65536, weights=True),
        # one sequence's cache cut to a budget
        _case("evict 32K to 4K", "evict", paged=False, n_lo=32768, n_hi=32768, sinks=4, recent=256),
        # a batch's paged caches cut to an eighth, with FP8 projections and gate terms
        _case("evict b16 8K-128K", "evict", B=16, n_lo=8192, n_hi=131072, sinks=4, recent=512, fp8=True, gate=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "chunk", "window", "evict"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    c = dict(op=op, B=_log_int(rng, 1, 24), Hq=Hkv * G, Hkv=Hkv, d=d, r=rng.choice([16, 32, 64]), paged=rng.random() < 0.6,
             fp8=rng.random() < 0.4, n_lo=1, n_hi=1, t_lo=1, t_hi=1, window=0, sinks=0, weights=False, keep_div=8,
             recent=0, fused=False, gate=False, pad=0)
    c["n_hi"] = _log_int(rng, 1, 32768 if op == "chunk" else 98304)
    c["n_hi"] = max(1, min(c["n_hi"], 700000 // c["B"]))
    if op in ("append", "chunk"):
        c["t_hi"] = min(c["n_hi"], _log_int(rng, 1, 4096))
        if op == "chunk":  # the plain form holds every score of the padded batch
            c["t_hi"] = max(1, min(c["t_hi"], int(1.0e9 / (c["B"] * c["Hq"] * c["n_hi"]))))
        else:
            c["t_hi"] = max(1, min(c["t_hi"], 16384 // c["B"]))
        c["t_lo"] = rng.choice([0, 1, c["t_hi"]])
        c["fused"] = rng.random() < 0.5
        c["pad"] = rng.choice([0, 0, 1, 7])
    c["n_lo"] = max(c["t_hi"], rng.choice([1, (c["n_hi"] + 1) // 2, c["n_hi"]]))
    if op in ("chunk", "window") and rng.random() < 0.6:
        c["window"] = _log_int(rng, 1, 8192)
        c["sinks"] = rng.choice([0, 1, 4, 64, 100])
    if op == "window":
        c["weights"] = rng.random() < 0.5
    if op == "evict":
        c["keep_div"] = rng.choice([1, 2, 4, 8, 32])
        c["sinks"] = rng.choice([0, 1, 4, 64])
        c["recent"] = rng.choice([0, 1, 64, 777])
        c["gate"] = rng.random() < 0.4
    return c


def _spread(lo, hi, n, step):
    """n whole numbers in [lo, hi], the ends among them, spread by a fixed rule of the case alone."""
    if n == 1:
        return [hi]
    v = [lo + int((hi - lo) * ((i * step) % 1.0)) for i in range(n)]
    v[0], v[-1] = hi, lo
    return v


def _sizes(c):
    """Cached tokens and new tokens of each sequence; the cache's capacity in rows."""
    lens = _spread(c["n_lo"], c["n_hi"], c["B"], 0.6180339887)
    new = _spread(c["t_lo"], c["t_hi"], c["B"], 0.7548776662) if c["op"] in ("append", "chunk") else [1] * c["B"]
    cap = -(-max(lens) // PAGE) * PAGE if c["paged"] else -(-max(lens) // 4) * 4
    return lens, new, cap


def _keep(c, lens):
    return [-(-n // c["keep_div"]) for n in lens]


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    B, Hq, Hkv, d, r = c["B"], c["Hq"], c["Hkv"], c["d"], c["r"]
    lens, new, cap = _sizes(c)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    s = dict(c, lens=lens, cap=cap)
    if c["paged"]:
        need = [-(-n // PAGE) for n in lens]
        num = sum(need)
        perm = torch.randperm(num, generator=g, device=dev).to(torch.int32)
        table = torch.full((B, cap // PAGE), -1, dtype=torch.int32, device=dev)
        at = 0
        for b in range(B):
            table[b, : need[b]] = perm[at: at + need[b]]
            at += need[b]
        s["page_table"], s["num_pages"] = table, num
        rows = (num, Hkv, PAGE)
    else:
        s["page_table"], s["num_pages"] = None, 0
        rows = (B, Hkv, cap)
    # keys with a decaying channel spectrum, as the workloads have them
    spectrum = torch.tensor([0.97 ** j for j in range(d)], device=dev)
    s["K"] = torch.empty(*rows, d, dtype=torch.bfloat16, device=dev)
    s["V"] = torch.empty(*rows, d, dtype=torch.bfloat16, device=dev)
    flat_k, flat_v = s["K"].view(-1, d), s["V"].view(-1, d)
    for i in range(0, flat_k.shape[0], 1 << 22):
        n = min(1 << 22, flat_k.shape[0] - i)
        flat_k[i: i + n] = torch.randn(n, d, generator=g, device=dev) * spectrum
        flat_v[i: i + n] = torch.randn(n, d, generator=g, device=dev)
    s["seqlens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if c["op"] in ("append", "evict"):
        basis = torch.linalg.qr(torch.randn(Hkv, d, d, generator=g, device=dev, dtype=torch.float64))[0]
        s["M"] = basis[:, :r, :].float().contiguous()
        s["Kproj"] = normal(*rows, r)
        s["scale"] = None
        if c["fp8"]:
            s["Kproj"] = s["Kproj"].float().to(torch.float8_e4m3fn)
            s["scale"] = torch.full((Hkv,), 2.0 ** -4, device=dev)
    if c["op"] in ("append", "chunk"):
        starts = [0]
        for t in new:
            starts.append(starts[-1] + t)
        total = starts[-1] + c["pad"]  # rows behind the last sequence belong to nobody
        s["q_start"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        s["n_new"], s["t_max"] = total, max(1, max(new))
        if c["fused"]:  # the rows of a fused projection: q, then k, then v
            x = normal(total, (Hq + 2 * Hkv) * d)
            s["q"] = x[:, : Hq * d].unflatten(1, (Hq, d))
            s["k_new"] = x[:, Hq * d: (Hq + Hkv) * d].unflatten(1, (Hkv, d))
            s["v_new"] = x[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d))
        else:
            s["q"] = normal(total, Hq, d)
            s["k_new"], s["v_new"] = normal(total, Hkv, d), normal(total, Hkv, d)
        if c["op"] == "chunk":
            s["out"] = torch.zeros(total, Hq, d, dtype=torch.bfloat16, device=dev)
            s["lse"] = torch.zeros(total, Hq, device=dev)
    if c["op"] == "window":
        s["q"] = normal(B, Hq, d)
        s["out"] = torch.zeros(B, Hq, d, device=dev)
        s["lse"] = torch.zeros(B, Hq, device=dev)
        s["acc"] = torch.rand(B, Hkv, cap, generator=g, device=dev) * 1e-3 if c["weights"] else None
    if c["op"] == "evict":
        # heavy-tailed weights: a few tokens hold most of the attention
        s["acc"] = torch.randn(B, Hkv, cap, generator=g, device=dev).mul_(2.0).exp_()
        keep = _keep(c, lens)
        s["keep"], s["keep_max"] = torch.tensor(keep, dtype=torch.int32, device=dev), max(1, max(keep))
        s["log_g"] = -torch.rand(B, Hkv, cap, generator=g, device=dev) * 12 if c["gate"] else None
        s["acc_out"] = torch.zeros(B, Hkv, cap, device=dev)
        s["idx"] = torch.zeros(B, Hkv, s["keep_max"], dtype=torch.int32, device=dev)
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _places(s, b, pos):
    """Cache coordinates (first, third axis) of positions `pos` of sequences `b` (same shapes)."""
    if s["page_table"] is None:
        return b, pos
    return s["page_table"][b, pos // PAGE].long(), pos % PAGE


def _rows(s, cache, pos, ok):
    """Rows [B][Hkv][n][...] of a cache in 32 bits at positions pos [B][n]; zeros where not ok."""
    b = torch.arange(s["B"], device=pos.device)[:, None].expand_as(pos)
    first, third = _places(s, b, torch.where(ok, pos, torch.zeros_like(pos)))
    if s["page_table"] is not None:
        first = first.clamp(min=0)
    x = cache[first, :, third].float()  # [B][n][Hkv][...]
    return torch.where(ok[:, :, None, None], x, torch.zeros_like(x)).transpose(1, 2)


def _tokens(s):
    """Sequence and position of every new token, and whether it belongs to a sequence."""
    t = torch.arange(s["n_new"], device=s["q_start"].device)
    start = s["q_start"].long()
    b = (torch.searchsorted(start, t, right=True) - 1).clamp(max=s["B"] - 1)
    pos = s["seqlens"].long()[b] - (start[b + 1] - start[b]) + t - start[b]
    return t, b, pos, t < start[-1]


def _plain_append(s):
    t, b, pos, ok = _tokens(s)
    t, b, pos = t[ok], b[ok], pos[ok]
    first, third = _places(s, b, pos)
    k, v = s["k_new"][t], s["v_new"][t]
    s["K"][first, :, third] = k
    s["V"][first, :, third] = v
    u = torch.einsum("thd,hrd->thr", k.double(), s["M"].double())
    if s["scale"] is not None:
        u = (u / s["scale"].double()[None, :, None]).clamp(-448, 448)
        s["Kproj"].view(torch.uint8)[first, :, third] = u.float().to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["Kproj"][first, :, third] = u.to(torch.bfloat16)
    return s


def _attend(q, k, v, visible, sigma):
    """q [..][m][d], k and v [..][n][d], visible [..][m][n]: output, log of the sum, weights."""
    z = torch.matmul(q, k.transpose(-1, -2)).mul_(sigma)
    z.masked_fill_(~visible, -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = z.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, v) / total
    return out, (total.log() + top).squeeze(-1), e, total


def _plain_chunk(s):
    B, Hkv, G, d = s["B"], s["Hkv"], s["Hq"] // s["Hkv"], s["d"]
    dev = s["q"].device
    start, lens = s["q_start"].long(), s["seqlens"].long()
    count = start[1:] - start[:-1]
    step = torch.arange(s["t_max"], device=dev)
    real = step[None, :] < count[:, None]                                    # [B][T]
    at = torch.where(real, start[:-1, None] + step[None, :], torch.zeros_like(real, dtype=torch.long))
    p = (lens - count)[:, None] + step[None, :]                              # positions
    q = s["q"][at].float().unflatten(2, (Hkv, G)).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)
    j = torch.arange(s["cap"], device=dev)[None, :].expand(B, -1)
    ok = j < lens[:, None]
    k, v = _rows(s, s["K"], j, ok), _rows(s, s["V"], j, ok)
    see = (j[:, None, :] <= p[:, :, None]) & real[:, :, None]                # [B][T][N]
    if s["window"]:
        see = see & ((j[:, None, :] > p[:, :, None] - s["window"]) | (j[:, None, :] < s["sinks"]))
    see = see.repeat_interleave(G, 1)[:, None]
    out, lse, _, _ = _attend(q, k, v, see, 1.0 / math.sqrt(d))
    out = out.unflatten(2, (-1, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)      # [B][T][Hq][d]
    lse = lse.unflatten(2, (-1, G)).permute(0, 2, 1, 3).flatten(2, 3)
    s["out"][at[real]] = out[real].to(torch.bfloat16)
    s["lse"][at[real]] = lse[real]
    return s


def _plain_window(s):
    B, Hkv, G, d = s["B"], s["Hkv"], s["Hq"] // s["Hkv"], s["d"]
    lens = s["seqlens"].long()
    if s["window"] and s["window"] + s["sinks"] < s["cap"]:  # only the rows that can be seen are read
        first = (lens - s["window"]).clamp(min=0)[:, None]
        a = torch.arange(s["sinks"], device=lens.device)[None, :].expand(B, -1)
        w = first + torch.arange(s["window"], device=lens.device)[None, :]
        j = torch.cat([a, w], 1)
        ok = torch.cat([a < torch.minimum(first, lens[:, None]), w < lens[:, None]], 1)
    else:
        j = torch.arange(s["cap"], device=lens.device)[None, :].expand(B, -1)
        ok = j < lens[:, None]
        if s["window"]:
            ok = ok & ((j > lens[:, None] - 1 - s["window"]) | (j < s["sinks"]))
    q = s["q"].float().view(B, Hkv, G, d)
    k, v = _rows(s, s["K"], j, ok), _rows(s, s["V"], j, ok)
    out, lse, e, total = _attend(q, k, v, ok[:, None, None, :], 1.0 / math.sqrt(d))
    s["out"].copy_(out.reshape(B, -1, d))
    s["lse"].copy_(lse.reshape(B, -1))
    if s["acc"] is not None:
        w = (e / total).sum(2) * ok[:, None, :]
        s["acc"].scatter_add_(2, torch.where(ok, j, torch.zeros_like(j))[:, None, :].expand_as(w), w)
    return s


def _plain_evict(s):
    B, Hkv = s["B"], s["Hkv"]
    lens, keep = s["seqlens"].long()[:, None, None], s["keep"].long()[:, None, None]
    n = torch.minimum(lens, keep)                                             # rows left
    j = torch.arange(s["cap"], device=lens.device)[None, None, :]
    rank = s["acc"].double()
    rank = torch.where(j >= lens - s["recent"], 1e300 + j.double() * 1e290, rank)
    rank = torch.where(j < s["sinks"], math.inf, rank)
    rank = torch.where(j < lens, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., : s["keep_max"]]
    o = torch.arange(s["keep_max"], device=lens.device)[None, None, :].expand(B, Hkv, -1)
    left = o < n
    idx = torch.sort(torch.where(left, order, s["cap"]), dim=-1)[0]
    s["idx"].copy_(torch.where(left, idx, -1))
    b = torch.arange(B, device=lens.device)[:, None, None].expand_as(idx)[left]
    h = torch.arange(Hkv, device=lens.device)[None, :, None].expand_as(idx)[left]
    src1, src3 = _places(s, b, idx[left])
    dst1, dst3 = _places(s, b, o[left])
    move = lambda x: x.index_put_((dst1, h, dst3), x[src1, h, src3])  # noqa: E731
    move(s["K"])
    move(s["V"])
    move(s["Kproj"].view(torch.uint8) if s["fp8"] else s["Kproj"])
    if s["log_g"] is not None:
        s["log_g"].index_put_((b, h, o[left]), s["log_g"][b, h, idx[left]])
    w = s["acc"][b, h, idx[left]]
    s["acc_out"].masked_fill_(j < lens, 0.0)
    s["acc_out"].index_put_((b, h, o[left]), w)
    s["new_lens"].copy_(n.flatten())
    return s


# ------------------------------------------------------------------------------------ the library's calls
def _session(s):
    if "session" not in s:  # kept by a user's program beside its caches
        from token_level_sparse_head_b200 import DecodeSession, Shape

        shape = Shape(s["B"], s["Hq"], s["Hkv"], s["d"], s["r"], 0 if s["paged"] else s["cap"], PAGE if s["paged"] else 0,
                      s["cap"] // PAGE if s["paged"] else 0, s["num_pages"], 1 if s["fp8"] and "scale" in s else 0, s.get("scale"))
        s["session"] = DecodeSession(shape, s.get("keep_max", 1), dense=False, chunk=s["n_new"] if s["op"] == "chunk" else 0,
                                     window=s["op"] == "window", weights=s["weights"], evict=s["op"] == "evict")
    return s["session"]


def _own(s):
    x = _session(s)
    if s["op"] == "append":
        x.append_chunk(s["k_new"], s["v_new"], s["q_start"], s["M"], s["K"], s["V"], s["Kproj"], s["page_table"], s["seqlens"])
    elif s["op"] == "chunk":
        x.chunk(s["q"], s["q_start"], s["K"], s["V"], s["page_table"], s["seqlens"], s["window"], s["sinks"], out=s["out"], lse=s["lse"])
    elif s["op"] == "window":
        x.window(s["q"], s["K"], s["V"], s["page_table"], s["seqlens"], s["window"], s["sinks"], weights=s["acc"], out=s["out"], lse=s["lse"])
    else:
        x.evict(s["acc"], s["keep"], s["sinks"], s["recent"], s["K"], s["V"], s["Kproj"], s["log_g"], s["page_table"], s["seqlens"],
                idx=s["idx"], weights_out=s["acc_out"], seqlens_out=s["new_lens"])
    return s


def _values(s):
    """The projected cache as the values that its codes stand for (exact in bf16: the scale is a power of two)."""
    if not s["fp8"]:
        return s["Kproj"]
    return (s["Kproj"].to(torch.bfloat16) * s["scale"].to(torch.bfloat16)[None, :, None, None])


def run(state):
    if own:
        s = _own(state)
    else:
        s = {"append": _plain_append, "chunk": _plain_chunk, "window": _plain_window, "evict": _plain_evict}[state["op"]](state)
    if s["op"] == "append":
        return {"K": s["K"], "V": s["V"], "Kproj": _values(s)}
    if s["op"] == "chunk":
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "window":
        return {"out": s["out"], "lse": s["lse"], "weights": s["acc"]}
    return {"K": s["K"], "V": s["V"], "Kproj": _values(s), "log_g": s["log_g"], "weights": s["acc_out"], "idx": s["idx"],
            "seqlens": s["new_lens"]}


# ------------------------------------------------------------------------------------ exact values
def _seen(p, n, window, sinks):
    """Positions that position p sees among n, as a list of ranges."""
    first = max(0, p - window + 1) if window else 0
    return [(0, min(sinks, first)), (first, min(p + 1, n))]


def _cache_index(s, b, pos):
    if s["page_table"] is None:
        return torch.full_like(pos, b), pos
    return s["page_table"][b].long()[pos // PAGE], pos % PAGE


def exact(case, seed):
    s = prepare(case, seed)
    lens, new, cap = _sizes(case)
    G, sigma = s["Hq"] // s["Hkv"], s["d"] ** -0.5
    dev = s["K"].device
    if s["op"] == "append":
        K, V, P = s["K"].double(), s["V"].double(), _values(s).double()
        at = 0
        for b, (n, t) in enumerate(zip(lens, new)):
            i1, i3 = _cache_index(s, b, torch.arange(n - t, n, device=dev))
            x = s["k_new"][at: at + t].double()
            for h in range(s["Hkv"]):
                K[i1, h, i3] = x[:, h]
                V[i1, h, i3] = s["v_new"][at: at + t, h].double()
                u = x[:, h] @ s["M"][h].double().T
                if s["scale"] is not None:  # E4M3: 3 fraction bits, steps of 2^-9 below 2^-6, at most 448
                    u = (u / s["scale"][h].double()).clamp(-448.0, 448.0)
                    step = torch.exp2((torch.frexp(u)[1] - 4).clamp(min=-9).double())
                    u = torch.round(u / step) * step * s["scale"][h].double()
                P[i1, h, i3] = u
            at += t
        return {"K": K, "V": V, "Kproj": P}
    if s["op"] == "chunk":
        out = torch.zeros(s["n_new"], s["Hq"], s["d"], dtype=torch.float64, device=dev)
        lse = torch.zeros(s["n_new"], s["Hq"], dtype=torch.float64, device=dev)
        at = 0
        for b, (n, t) in enumerate(zip(lens, new)):
            i1, i3 = _cache_index(s, b, torch.arange(n, device=dev))
            for t0 in range(0, t, 512):
                t1 = min(t, t0 + 512)
                p = torch.arange(n - t + t0, n - t + t1, device=dev)[:, None]
                j = torch.arange(n, device=dev)[None, :]
                hide = j > p
                if s["window"]:
                    hide |= (j <= p - s["window"]) & (j >= s["sinks"])
                for h in range(s["Hkv"]):
                    k, v = s["K"][i1, h, i3].double(), s["V"][i1, h, i3].double()
                    for g in range(h * G, (h + 1) * G):
                        z = (s["q"][at + t0: at + t1, g].double() @ k.T) * sigma
                        z[hide] = -math.inf
                        lse[at + t0: at + t1, g] = torch.logsumexp(z, -1)
                        out[at + t0: at + t1, g] = torch.softmax(z, -1) @ v
            at += t
        return {"out": out, "lse": lse}
    if s["op"] == "window":
        out = torch.zeros(s["B"], s["Hq"], s["d"], dtype=torch.float64, device=dev)
        lse = torch.zeros(s["B"], s["Hq"], dtype=torch.float64, device=dev)
        acc = None if s["acc"] is None else s["acc"].double()
        for b, n in enumerate(lens):
            pos = torch.cat([torch.arange(x, y, device=dev) for x, y in _seen(n - 1, n, s["window"], s["sinks"])])
            i1, i3 = _cache_index(s, b, pos)
            for h in range(s["Hkv"]):
                z = (s["q"][b, h * G:(h + 1) * G].double() @ s["K"][i1, h, i3].double().T) * sigma
                w = torch.softmax(z, -1)
                out[b, h * G:(h + 1) * G] = w @ s["V"][i1, h, i3].double()
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
                if acc is not None:
                    acc[b, h, pos] += w.sum(0)
        return {"out": out, "lse": lse, "weights": acc}
    import numpy as np

    idx = np.full((s["B"], s["Hkv"], s["keep_max"]), -1, dtype=np.int64)
    K, V, P = s["K"].double(), s["V"].double(), _values(s).double()
    gate = None if s["log_g"] is None else s["log_g"].double()
    acc = torch.zeros(s["B"], s["Hkv"], cap, dtype=torch.float64, device=dev)
    keep = _keep(case, lens)
    for b, n in enumerate(lens):
        for h in range(s["Hkv"]):
            w = s["acc"][b, h, :n].cpu().numpy().astype(np.float64)
            tier = np.zeros(n, dtype=np.int64)
            tier[max(0, n - s["recent"]):] = np.arange(1, n - max(0, n - s["recent"]) + 1)
            tier[: s["sinks"]] = n + 1
            best = np.sort(np.lexsort((np.arange(n), -np.where(tier > 0, 0.0, w), -tier))[: keep[b]])
            idx[b, h, : len(best)] = best
            src = torch.from_numpy(best).to(dev)
            i1, i3 = _cache_index(s, b, src)
            o1, o3 = _cache_index(s, b, torch.arange(len(best), device=dev))
            for x in (K, V, P):
                x[o1, h, o3] = x[i1, h, i3].clone()
            if gate is not None:
                gate[b, h, : len(best)] = gate[b, h, src].clone()
            acc[b, h, : len(best)] = s["acc"][b, h, src].double()
    return {"K": K, "V": V, "Kproj": P, "log_g": gate, "weights": acc, "idx": torch.from_numpy(idx).to(torch.int32),
            "seqlens": torch.tensor([min(n, k) for n, k in zip(lens, keep)], dtype=torch.int32)}


# ------------------------------------------------------------------------------------ the least work
def work(case):
    c = case
    lens, new, cap = _sizes(c)
    kv, es = 4.0 * c["d"], 1.0 if c["fp8"] else 2.0
    if c["op"] == "append":
        n = float(sum(new)) * c["Hkv"]
        return {"bytes": n * (2 * kv + c["r"] * es) + c["Hkv"] * c["r"] * c["d"] * 4.0, "flops": n * 2.0 * c["r"] * c["d"]}
    if c["op"] == "evict":
        keep = _keep(c, lens)
        moved = float(sum(min(n, k) for n, k in zip(lens, keep))) * c["Hkv"]
        row = kv + c["r"] * es + 4.0 + (4.0 if c["gate"] else 0.0)
        return {"bytes": sum(lens) * c["Hkv"] * 4.0 + moved * (2 * row + 4.0), "flops": 0.0}
    rows = pairs = toks = 0.0
    for n, t in zip(lens, new):
        if t == 0:
            continue
        toks += t
        rows += sum(y - x for x, y in _seen(n - t, n, c["window"], c["sinks"])) + (t - 1)
        for p in range(n - t, n):
            pairs += sum(y - x for x, y in _seen(p, n, c["window"], c["sinks"]))
    out = 2.0 if c["op"] == "chunk" else 4.0
    moved = toks * c["Hq"] * (c["d"] * (2.0 + out) + 4.0) + rows * c["Hkv"] * kv
    if c["weights"]:
        moved += rows * c["Hkv"] * 8.0
    return {"bytes": moved, "flops": 4.0 * c["d"] * c["Hq"] * pairs}
