"""Measured cases of the serving operators that surround the attention calls of this library:
packed prompts (fwd_varlen, fwd_varlen_paged), rotary positions with several axes (rope,
rope_append), filling a paged cache (cache_append, rope_append) and managing its pages
(pages_free, pages_fork, pages_reserve, pages_compact, pages_copy).

Every operator is also written here in plain torch operations, in 32 bits (angles in 64),
rounded once at the end; `own` selects between that and the library's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
NEG = float("-inf")


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # a few short chat turns arriving at once: latency counts
        dict(name="varlen-short", op="varlen", B=8, lo=1, hi=64, Hq=32, Hkv=8, d=128, causal=True, window=0, cross=False, seed=3),
        # an ordinary packed batch of prompts, read from one fused projection buffer
        dict(name="varlen-ragged", op="varlen", B=16, lo=16, hi=2048, Hq=32, Hkv=8, d=128, causal=True, window=0, cross=False, seed=5),
        # long documents beside short questions
        dict(name="varlen-long", op="varlen", B=9, lo=500, hi=8192, Hq=32, Hkv=8, d=128, causal=True, window=0, cross=False, seed=8),
        # three query heads to a key head, head dim 64, a sliding window, more keys than queries
        dict(name="varlen-window-d64", op="varlen", B=13, lo=33, hi=3001, Hq=12, Hkv=4, d=64, causal=True, window=512, cross=True, seed=13),
        # chunks of prompts that continue contexts held in cache pages
        dict(name="varlen-paged", op="paged", B=12, lo=1, hi=512, ctx=8192, page=64, Hq=32, Hkv=8, d=128, window=0, seed=21),
        # one decode step of an image-and-text model: three position axes
        dict(name="rope-decode", op="rope", T=32, Hq=32, Hkv=8, d=128, F=64, A=3, inter=False, inverse=False, dtype="bf16", far=1 << 20),
        # the prompt of the same model
        dict(name="rope-prompt", op="rope", T=16384, Hq=32, Hkv=8, d=128, F=64, A=3, inter=False, inverse=False, dtype="bf16", far=32768),
        # the gradient of a partial, adjacent-pair rotation kept in 32 bits, odd length
        dict(name="rope-gradient", op="rope", T=4095, Hq=16, Hkv=2, d=128, F=32, A=1, inter=True, inverse=True, dtype="fp32", far=8192),
        # one decode step: rotate q and k, put k and v into the pages
        dict(name="append-decode", op="append", B=32, lo=1, hi=1, ctx=1024, page=64, Hq=32, Hkv=8, d=128, rope=True, fp8=False, A=1),
        # a packed batch of prompts encoded into an FP8 cache
        dict(name="append-prompt-fp8", op="append", B=16, lo=100, hi=2048, ctx=0, page=64, Hq=32, Hkv=8, d=128, rope=False, fp8=True, A=1),
        # several answers sampled from each cached prompt: drop the last ones, fork, extend, copy the split pages
        dict(name="pages-sample", op="pages", parents=8, kids=7, ctx=2048, add=1, page=64, Hkv=8, d=128),
        # defragmenting a pool after many requests have ended
        dict(name="pages-compact", op="compact", S=64, pages=2048, live=0.55, page=64, Hkv=8, d=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["varlen", "varlen", "paged", "rope", "append", "pages", "compact"])
    seed = rng.randrange(1 << 20)
    Hq, Hkv = rng.choice([(32, 8), (8, 2), (12, 4), (8, 8), (16, 1), (6, 2)])
    d = rng.choice([64, 128])
    if kind == "varlen":
        B = _log(rng, 1, 32)
        hi = _log(rng, 8, max(8, min(8192, 24000 // B)))
        causal = rng.random() < 0.75
        return dict(op=kind, B=B, lo=max(1, hi // rng.choice([2, 8, 64])), hi=hi, Hq=Hq, Hkv=Hkv, d=d, causal=causal,
                    window=rng.choice([0, 0, _log(rng, 1, 4000)]) if causal else 0, cross=rng.random() < 0.3, seed=seed)
    if kind == "paged":
        return dict(op=kind, B=_log(rng, 1, 12), lo=1, hi=_log(rng, 1, 500), ctx=_log(rng, 1, 8000),
                    page=rng.choice([16, 48, 64, 128]), Hq=Hq, Hkv=Hkv, d=d, window=rng.choice([0, 0, _log(rng, 1, 3000)]),
                    seed=seed)
    if kind == "rope":
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        return dict(op=kind, T=_log(rng, 1, 8192 if dtype == "fp32" else 16000), Hq=Hq, Hkv=Hkv, d=d,
                    F=rng.choice([d // 2, d // 2, d // 4, 12]), A=rng.choice([1, 2, 3]), inter=rng.random() < 0.5,
                    inverse=rng.random() < 0.5, dtype=dtype, far=_log(rng, 1000, 1 << 22))
    if kind == "append":
        fp8, hi = rng.random() < 0.5, _log(rng, 1, 1500)
        return dict(op=kind, B=_log(rng, 1, 32 if hi < 500 else 12), lo=1, hi=hi, ctx=_log(rng, 1, 1000),
                    page=rng.choice([16, 48, 64, 128]), Hq=Hq, Hkv=Hkv, d=128 if fp8 else d, rope=not fp8, fp8=fp8,
                    A=rng.choice([1, 3]))
    if kind == "pages":
        return dict(op=kind, parents=_log(rng, 1, 16), kids=rng.randint(1, 8), ctx=_log(rng, 1, 3000),
                    add=_log(rng, 1, 200), page=rng.choice([16, 48, 64, 128]), Hkv=rng.choice([1, 2, 8]), d=d)
    return dict(op=kind, S=_log(rng, 1, 64), pages=_log(rng, 64, 2000), live=round(rng.uniform(0.05, 0.95), 3),
                page=rng.choice([16, 32, 64]), Hkv=rng.choice([1, 2, 8]), d=d)


# ------------------------------------------------------------------------------ inputs

def _lengths(case):
    """The lengths belong to the case: its work does not depend on the inputs' seed."""
    r = np.random.RandomState(case.get("seed", 7))
    lo, hi, B = case["lo"], case["hi"], case["B"]
    n = np.exp(r.uniform(math.log(lo), math.log(hi + 0.999), B)).astype(np.int64).clip(lo, hi)
    n[0] = hi
    return n


def _contexts(case):
    r = np.random.RandomState(case.get("seed", 7) + 1)
    return r.randint(0, case["ctx"] + 1, case["B"]) if case["ctx"] else np.zeros(case["B"], np.int64)


def _keys(case, nq):
    """Keys of each sequence: as many as queries, or some cached ones before them."""
    if not case["cross"]:
        return nq
    return nq + np.random.RandomState(case["seed"] + 2).randint(0, max(1, case["hi"] // 2), case["B"])


def _cu(n):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(DEV)


def _gen(seed):
    return torch.Generator(DEV).manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _tables(pages_per_seq, spare, seed):
    """A block table whose pages lie scattered over the pool, -1 behind them, and the refcounts."""
    n = np.asarray(pages_per_seq)
    total = int(n.sum()) + spare
    perm = np.random.RandomState(int(seed) & 0x7FFFFFFF).permutation(total)
    table = np.full((len(n), max(1, int(n.max()))), -1, np.int32)
    ref = np.zeros(total, np.int32)
    at = 0
    for s, m in enumerate(n):
        table[s, :m] = perm[at:at + m]
        ref[perm[at:at + m]] = 1
        at += m
    return table, ref, total


def _pool(g, pages, Hkv, page, d, fp8=False):
    x = _randn(g, pages, Hkv, page, d)
    return x.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else x


def _positions(g, case, T):
    far = case.get("far", 32768)
    return torch.randint(0, far, (case["A"], T), generator=g, device=DEV, dtype=torch.int32)


def _freqs(case, F):
    inv = (10000.0 ** (-np.arange(F) / F)).astype(np.float32)
    axes = (np.arange(F) * case["A"] // F).astype(np.int32)  # contiguous sections, one for each axis
    return torch.from_numpy(inv).to(DEV), torch.from_numpy(axes).to(DEV)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("varlen", "paged"):
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
        nq = _lengths(case)
        Tq = int(nq.sum())
        if op == "varlen":
            nk = _keys(case, nq)
            Tk = int(nk.sum())
            if Tk == Tq:  # slices of one projection's output
                qkv = _randn(g, Tq, Hq + 2 * Hkv, d)
                s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
            else:
                s["q"], s["k"], s["v"] = _randn(g, Tq, Hq, d), _randn(g, Tk, Hkv, d), _randn(g, Tk, Hkv, d)
            s["cu_k"] = _cu(nk)
        else:
            nk = nq + _contexts(case)
            table, _, total = _tables(-(-nk // case["page"]), 5, seed)
            s["q"] = _randn(g, Tq, Hq, d)
            s["kp"], s["vp"] = (_pool(g, total, Hkv, case["page"], d) for _ in range(2))
            s["table"] = torch.from_numpy(table).to(DEV)
            s["seqlens"] = torch.from_numpy(nk.astype(np.int32)).to(DEV)
        s["nq"], s["nk"], s["cu_q"] = nq.tolist(), nk.tolist(), _cu(nq)
        s["out"] = torch.empty(Tq, Hq, d, device=DEV, dtype=torch.bfloat16)
        s["lse"] = torch.empty(Hq, Tq, device=DEV, dtype=torch.float32)
        # scratch that a program keeps for all its calls
        s["ws"] = torch.empty(32 * (Tq // 128 + 2 * len(nq) + 64) + 65536, device=DEV, dtype=torch.uint8)
    elif op == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        T = case["T"]
        s["q"], s["k"] = _randn(g, T, case["Hq"], case["d"], dtype=dt), _randn(g, T, case["Hkv"], case["d"], dtype=dt)
        s["pos"] = _positions(g, case, T)
        s["inv"], s["axes"] = _freqs(case, case["F"])
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    elif op == "append":
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
        n = _lengths(case)
        T = int(n.sum())
        lens = n + _contexts(case)
        table, _, total = _tables(-(-lens // case["page"]), 3, seed)
        s["q"], s["k"], s["v"] = _randn(g, T, Hq, d), _randn(g, T, Hkv, d), _randn(g, T, Hkv, d)
        s["q_out"] = torch.empty_like(s["q"])
        s["kp"], s["vp"] = (_pool(g, total, Hkv, case["page"], d, case["fp8"]) for _ in range(2))
        s["table"] = torch.from_numpy(table).to(DEV)
        s["cu"], s["seqlens"] = _cu(n), torch.from_numpy(lens.astype(np.int32)).to(DEV)
        s["ks"], s["vs"] = (torch.rand(Hkv, generator=g, device=DEV) * 0.01 + 0.005 for _ in range(2))
        s["pos"] = _positions(g, case, T)
        s["inv"], s["axes"] = _freqs(case, d // 2)
    elif op == "pages":
        P, K, page = case["parents"], case["kids"], case["page"]
        lens = np.zeros(P * (K + 1), np.int64)
        lens[:P] = np.random.RandomState(11).randint(1, case["ctx"] + 1, P)
        table, ref, total = _tables(-(-lens // page), P * K * (2 + case["add"] // page) + 4, seed)
        grown = -(-(int(lens.max()) + case["add"]) // page)
        wide = np.full((len(lens), grown), -1, np.int32)
        wide[:, :table.shape[1]] = table
        s["table"], s["ref"] = torch.from_numpy(wide).to(DEV), torch.from_numpy(ref).to(DEV)
        s["seqlens"] = torch.from_numpy(lens.astype(np.int32)).to(DEV)
        kids = np.arange(P, P * (K + 1), dtype=np.int32)
        src = np.repeat(np.arange(P, dtype=np.int32), K)
        add = np.zeros(len(lens), np.int32)
        add[P:] = case["add"]
        s["dst"], s["src"], s["add"] = (torch.from_numpy(x).to(DEV) for x in (kids, src, add))
        s["copied"] = torch.from_numpy(np.flatnonzero(lens[src] % page) + P).to(DEV)  # slots whose last page splits
        s["copies"] = torch.empty(len(lens), 2, device=DEV, dtype=torch.int32)
        s["ws"] = torch.empty(4 * (total + len(lens)) + 4096, device=DEV, dtype=torch.uint8)
        s["kp"], s["vp"] = (_pool(g, total, case["Hkv"], page, case["d"]) for _ in range(2))
    else:
        N, S = case["pages"], case["S"]
        r = np.random.RandomState(17)
        live = max(1, min(N - 1, int(N * case["live"])))
        owner = np.sort(r.randint(0, S, live))
        counts = np.bincount(owner, minlength=S)
        table, ref, _ = _tables(counts, N - live, seed)
        s["table0"], s["ref0"] = torch.from_numpy(table).to(DEV), torch.from_numpy(ref).to(DEV)
        s["table"], s["ref"] = torch.empty_like(s["table0"]), torch.empty_like(s["ref0"])
        lens = np.maximum(counts * case["page"] - r.randint(0, case["page"], S) * (counts > 0), 0)
        s["seqlens"] = torch.from_numpy(lens.astype(np.int32)).to(DEV)
        s["moves"] = int((ref[live:] > 0).sum())
        s["copies"] = torch.empty(N // 2, 2, device=DEV, dtype=torch.int32)
        s["ws"] = torch.empty(8 * N + 4096, device=DEV, dtype=torch.uint8)
        s["kp"], s["vp"] = (_pool(g, N, case["Hkv"], case["page"], case["d"]) for _ in range(2))
    return s


# ------------------------------------------------------------------------- plain forms

def _attend(q, k, v, causal, window, scale):
    """One sequence: q (n,Hq,d), k and v (m,Hkv,d) in 32 bits -> o (n,Hq,d), lse (Hq,n)."""
    n, Hq, d = q.shape
    m, Hkv = k.shape[:2]
    s = torch.einsum("nhrd,mhd->hrnm", q.reshape(n, Hkv, Hq // Hkv, d), k) * scale
    if causal:
        i = torch.arange(n, device=DEV)[:, None] + (m - n)
        j = torch.arange(m, device=DEV)[None, :]
        hidden = j > i
        if window:
            hidden = hidden | (j <= i - window)
        s = s.masked_fill(hidden, NEG)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("hrnm,mhd->nhrd", p, v) / total.permute(2, 0, 1, 3)
    lse = (top + torch.log(total)).reshape(Hq, n)
    return o.reshape(n, Hq, d), lse


def _plain_packed(s, keys):
    """The sequences one after another (their scores do not fit as one padded tensor)."""
    c = s["case"]
    q, out, lse = s["q"], s["out"], s["lse"]
    scale, at = 1.0 / math.sqrt(c["d"]), 0
    for b, n in enumerate(s["nq"]):
        k, v = keys(b)
        o, l = _attend(q[at:at + n].float(), k.float(), v.float(), c.get("causal", True), c["window"], scale)
        out[at:at + n] = o.to(out.dtype)
        lse[:, at:at + n] = l
        at += n
    return out, lse


def _plain_rotate(x, pos, inv, axes, inter, inverse):
    F = inv.shape[0]
    ang = pos[axes.long()].double() * inv.double()[:, None]            # (F, T)
    cos, sin = torch.cos(ang).float().t()[:, None], torch.sin(ang).float().t()[:, None]
    if inverse:
        sin = -sin
    y = x.float()
    a, b = (y[..., 0:2 * F:2], y[..., 1:2 * F:2]) if inter else (y[..., :F], y[..., F:2 * F])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([u, w], -1).flatten(-2) if inter else torch.cat([u, w], -1)
    return torch.cat([turned, y[..., 2 * F:]], -1)


def _plain_append(s):
    c = s["case"]
    q, k, v = s["q"], s["k"].float(), s["v"].float()
    T, page = k.shape[0], c["page"]
    if c["rope"]:
        q = _plain_rotate(q, s["pos"], s["inv"], s["axes"], False, False).to(q.dtype)
        k = _plain_rotate(k, s["pos"], s["inv"], s["axes"], False, False)
    cu = s["cu"].long()
    i = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu, i, right=True) - 1
    at = s["seqlens"].long()[b] - cu[b + 1] + i
    pg, row = s["table"].long()[b, at // page], at % page
    if c["fp8"]:
        code = lambda x, sc: (x / sc[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        k, v = code(k, s["ks"]), code(v, s["vs"])
    s["kp"][pg, :, row] = k.to(s["kp"].dtype)
    s["vp"][pg, :, row] = v.to(s["vp"].dtype)
    return q, s["kp"], s["vp"]


def _plain_count(ref, table, keep, by):
    """ref + by for every table entry that `keep` marks."""
    return ref.index_add_(0, table.clamp(min=0).flatten().long(), keep.flatten().to(ref.dtype) * by)


def _plain_sample(s):
    c = s["case"]
    page, table, lens, ref = c["page"], s["table"], s["seqlens"], s["ref"]
    src, dst, add, copies = s["src"].long(), s["dst"].long(), s["add"], s["copies"]
    j = torch.arange(table.shape[1], device=DEV)
    _plain_count(ref, table[dst], table[dst] >= 0, -1)                  # free
    table[dst] = -1
    lens[dst] = lens[src]                                               # fork
    table[dst] = table[src]
    _plain_count(ref, table[src], table[src] >= 0, 1)
    old, new = (lens + page - 1) // page, (lens + add + page - 1) // page   # reserve
    last = table.gather(1, (old - 1).clamp(min=0).long()[:, None])[:, 0]
    split = (add > 0) & (lens % page > 0) & (ref[last.clamp(min=0).long()] > 1)
    need = new - old + split
    first = torch.cumsum(need, 0) - need
    free = ref == 0
    rank = torch.cumsum(free, 0) - 1
    ids = torch.empty(ref.shape[0] + 1, device=DEV, dtype=torch.int32)
    ids[torch.where(free, rank, ref.shape[0])] = torch.arange(ref.shape[0], device=DEV, dtype=torch.int32)
    begin = old - split.int()
    fresh = (j >= begin[:, None]) & (j < new[:, None])
    table.copy_(torch.where(fresh, ids[(first[:, None] + j - begin[:, None]).clamp(0, ref.shape[0]).long()], table))
    ref.index_add_(0, last.clamp(min=0).long(), -split.to(ref.dtype))
    _plain_count(ref, table, fresh, 1)
    lens += add
    moved = table.gather(1, begin.clamp(min=0, max=table.shape[1] - 1).long()[:, None])[:, 0]
    copies.copy_(torch.where(split[:, None], torch.stack([last, moved], 1), -1))
    at = copies[s["copied"]].long()                                     # copy
    s["kp"][at[:, 1]] = s["kp"][at[:, 0]]
    s["vp"][at[:, 1]] = s["vp"][at[:, 0]]
    return table, lens, ref, copies, s["kp"], s["vp"]


def _plain_compact(s):
    table, ref, copies, N = s["table"], s["ref"], s["copies"], s["ref"].shape[0]
    at = torch.arange(N, device=DEV, dtype=torch.int32)
    live = ref > 0
    n = live.sum()
    hole, mover = ~live & (at < n), live & (at >= n)
    holes, movers = (torch.empty(N + 1, device=DEV, dtype=torch.int32) for _ in range(2))
    holes[torch.where(hole, torch.cumsum(hole, 0) - 1, N)] = at
    rank = torch.cumsum(mover, 0) - 1
    movers[torch.where(mover, rank, N)] = at
    used = at[:copies.shape[0]] < mover.sum()
    copies.copy_(torch.where(used[:, None], torch.stack([movers, holes], 1)[:copies.shape[0]], -1))
    to = torch.where(mover, holes[rank.clamp(min=0)], at)
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
    moved = torch.zeros_like(ref).index_add_(0, to.long(), ref)
    ref.copy_(moved)
    go = copies[:s["moves"]].long()
    s["kp"][go[:, 1]] = s["kp"][go[:, 0]]
    s["vp"][go[:, 1]] = s["vp"][go[:, 0]]
    return table, ref, copies, s["kp"], s["vp"]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "varlen":
        at = np.concatenate([[0], np.cumsum(s["nk"])])
        return _plain_packed(s, lambda b: (s["k"][at[b]:at[b + 1]], s["v"][at[b]:at[b + 1]]))
    if op == "paged":
        def keys(b):
            n = s["nk"][b]
            pg = s["table"][b, :-(-n // c["page"])].long()
            return tuple(p[pg].transpose(1, 2).flatten(0, 1)[:n] for p in (s["kp"], s["vp"]))
        return _plain_packed(s, keys)
    if op == "rope":
        q, k = (_plain_rotate(x, s["pos"], s["inv"], s["axes"], c["inter"], c["inverse"]) for x in (s["q"], s["k"]))
        return s["q_out"].copy_(q), s["k_out"].copy_(k)
    if op == "append":
        q, kp, vp = _plain_append(s)
        return _appended(c, s["q_out"].copy_(q) if c["rope"] else None, kp, vp)
    if op == "pages":
        return _plain_sample(s)
    return _plain_compact(s)


def _appended(c, q, kp, vp):
    if c["fp8"]:  # the values that the bytes stand for
        return kp.view(torch.float8_e4m3fn), vp.view(torch.float8_e4m3fn)
    return q, kp, vp


def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if op == "compact":  # the fragmented tables again
        s["table"].copy_(s["table0"])
        s["ref"].copy_(s["ref0"])
    if not own:
        return _plain(s)
    from exact_io_aware_81_b200 import ops
    if op == "varlen":
        return ops.fwd_varlen(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=c["causal"], window=c["window"],
                              workspace=s["ws"], out=s["out"], lse=s["lse"])
    if op == "paged":
        return ops.fwd_varlen_paged(s["q"], s["kp"], s["vp"], s["table"], s["cu_q"], s["seqlens"], causal=True,
                                    window=c["window"], workspace=s["ws"], out=s["out"], lse=s["lse"])
    if op == "rope":
        return ops.rope(s["q"], s["k"], s["pos"], s["inv"], s["axes"], interleaved=c["inter"], inverse=c["inverse"],
                        q_out=s["q_out"], k_out=s["k_out"])
    if op == "append":
        if c["rope"]:
            ops.rope_append(s["q"], s["k"], s["v"], s["pos"], s["inv"], s["kp"], s["vp"], s["table"], s["cu"],
                            s["seqlens"], axes=s["axes"], q_out=s["q_out"])
        else:
            ops.cache_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["cu"], s["seqlens"], k_scale=s["ks"],
                             v_scale=s["vs"])
        return _appended(c, s["q_out"], s["kp"], s["vp"])
    if op == "pages":
        pool = (s["table"], s["seqlens"], s["ref"])
        ops.pages_free(*pool, s["dst"], c["page"])
        ops.pages_fork(*pool, s["src"], s["dst"], c["page"])
        ops.pages_reserve(*pool, s["add"], c["page"], copies=s["copies"], workspace=s["ws"])
        ops.pages_copy(s["kp"], s["vp"], s["copies"])
        return *pool, s["copies"], s["kp"], s["vp"]
    ops.pages_compact(s["table"], s["seqlens"], s["ref"], c["page"], copies=s["copies"], workspace=s["ws"])
    ops.pages_copy(s["kp"], s["vp"], s["copies"])
    return s["table"], s["ref"], s["copies"], s["kp"], s["vp"]


# -------------------------------------------------------------------------------- work

def work(case):
    op, c = case["op"], case
    if op in ("varlen", "paged"):
        nq = _lengths(c)
        nk = _keys(c, nq) if op == "varlen" else nq + _contexts(c)
        w = c["window"]
        seen = 0
        for n, m in zip(nq.tolist(), nk.tolist()):
            i = np.arange(n, dtype=np.int64) + (m - n) + 1  # keys up to the diagonal
            seen += int((np.minimum(i, w) if w else i).sum()) if c.get("causal", True) else n * m
        per = c["d"] * 2
        size = 2 * int(nq.sum()) * c["Hq"] * per + 2 * int(nk.sum()) * c["Hkv"] * per + 4 * int(nq.sum()) * c["Hq"]
        return {"bytes": size, "flops": 4 * c["d"] * c["Hq"] * seen}
    if op == "rope":
        e = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": c["T"] * (2 * (c["Hq"] + c["Hkv"]) * c["d"] * e + 4 * c["A"]),
                "flops": c["T"] * (c["Hq"] + c["Hkv"]) * 6 * c["F"]}
    if op == "append":
        T = int(_lengths(c).sum())
        e = 1 if c["fp8"] else 2
        size = T * 2 * c["Hkv"] * c["d"] * (2 + e) + (T * (2 * c["Hq"] * c["d"] * 2 + 4 * c["A"]) if c["rope"] else 0)
        return {"bytes": size, "flops": T * 2 * c["Hkv"] * c["d"]}
    one = 2 * c["page"] * c["Hkv"] * c["d"] * 2  # K and V of a page
    if op == "pages":
        lens = np.random.RandomState(11).randint(1, c["ctx"] + 1, c["parents"])
        pairs = int((lens % c["page"] > 0).sum()) * c["kids"]
        rows = c["kids"] * int((-(-lens // c["page"])).sum())
        return {"bytes": 2 * one * pairs + 16 * rows + 4 * c["parents"] * c["kids"], "flops": 0}
    live = max(1, min(c["pages"] - 1, int(c["pages"] * c["live"])))
    moves = live * (c["pages"] - live) // c["pages"]  # expected: live pages behind the first `live`
    return {"bytes": 2 * one * moves + 8 * c["pages"] + 8 * live, "flops": 0}


# ------------------------------------------------------------------------------- exact

def _exact_attention(q, k, v, causal, window):
    """Row blocks in 64 bits; every query head against its own key head."""
    n, Hq, d = q.shape
    m, Hkv = k.shape[:2]
    o = torch.empty(n, Hq, d, device=DEV, dtype=torch.float64)
    lse = torch.empty(Hq, n, device=DEV, dtype=torch.float64)
    cols = torch.arange(m, device=DEV)
    for h in range(Hq):
        kk, vv, qq = k[:, h * Hkv // Hq].double(), v[:, h * Hkv // Hq].double(), q[:, h].double()
        for r in range(0, n, 4096):
            t = (qq[r:r + 4096] @ kk.T) / math.sqrt(d)
            if causal:
                last = torch.arange(r, r + t.shape[0], device=DEV)[:, None] + m - n
                ok = cols <= last
                if window:
                    ok &= cols > last - window
                t = torch.where(ok, t, torch.full_like(t, NEG))
            z = torch.logsumexp(t, 1)
            o[r:r + 4096, h] = torch.exp(t - z[:, None]) @ vv
            lse[h, r:r + 4096] = z
    return o, lse


def _exact_rotation(x, pos, inv, axes, inter, inverse):
    y = x.double().clone()
    for f in range(inv.shape[0]):
        t = pos[int(axes[f])].double() * float(inv[f])
        z = torch.complex(torch.cos(t), -torch.sin(t) if inverse else torch.sin(t))
        i, j = (2 * f, 2 * f + 1) if inter else (f, f + inv.shape[0])
        w = torch.complex(x[..., i].double(), x[..., j].double()) * z[:, None]
        y[..., i], y[..., j] = w.real, w.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op in ("varlen", "paged"):
        os_, ls, a, b = [], [], 0, 0
        for i, (n, m) in enumerate(zip(s["nq"], s["nk"])):
            if op == "varlen":
                k, v = s["k"][b:b + m], s["v"][b:b + m]
            else:
                t = torch.arange(m, device=DEV)
                pg = s["table"][i].long()[t // c["page"]]
                k, v = s["kp"][pg, :, t % c["page"]], s["vp"][pg, :, t % c["page"]]
            o, l = _exact_attention(s["q"][a:a + n], k, v, c.get("causal", True), c["window"])
            os_.append(o)
            ls.append(l)
            a, b = a + n, b + m
        return torch.cat(os_), torch.cat(ls, 1)
    if op == "rope":
        return tuple(_exact_rotation(x, s["pos"], s["inv"], s["axes"], c["inter"], c["inverse"]) for x in (s["q"], s["k"]))
    if op == "append":
        q, k, v = s["q"], s["k"].double(), s["v"].double()
        kp, vp = ((p.view(torch.float8_e4m3fn) if c["fp8"] else p).double() for p in (s["kp"], s["vp"]))
        if c["rope"]:
            q, k = (_exact_rotation(x, s["pos"], s["inv"], s["axes"], False, False) for x in (q, k))
        if c["fp8"]:
            k, v = ((x / sc.double()[:, None]).clamp(-448, 448) for x, sc in ((k, s["ks"]), (v, s["vs"])))
        cu, lens, table = s["cu"].tolist(), s["seqlens"].tolist(), s["table"].long()
        for b in range(c["B"]):
            t = torch.arange(lens[b] - (cu[b + 1] - cu[b]), lens[b], device=DEV)
            kp[table[b][t // c["page"]], :, t % c["page"]] = k[cu[b]:cu[b + 1]]
            vp[table[b][t // c["page"]], :, t % c["page"]] = v[cu[b]:cu[b + 1]]
        return (kp, vp) if c["fp8"] else (q, kp, vp)
    kp, vp = s["kp"].double(), s["vp"].double()
    if op == "pages":
        ref, table, lens = s["ref"].cpu().numpy().copy(), s["table"].cpu().numpy(), s["seqlens"].tolist()
        free = iter(np.flatnonzero(ref == 0).tolist())
        for src in s["src"].tolist():  # the children's slots come in this order
            n = lens[src]
            if n % c["page"]:
                a, b = int(table[src, n // c["page"]]), next(free)
                kp[b], vp[b] = kp[a].clone(), vp[a].clone()
            for _ in range(-(-(n + c["add"]) // c["page"]) - (-(-n // c["page"]))):
                next(free)
        return None, None, None, None, kp, vp
    ref = s["ref0"].cpu().numpy()
    n = int((ref > 0).sum())
    for b, a in zip(np.flatnonzero(ref[:n] == 0).tolist(), (np.flatnonzero(ref[n:] > 0) + n).tolist()):
        kp[b], vp[b] = kp[a].clone(), vp[a].clone()
    return None, None, None, kp, vp
