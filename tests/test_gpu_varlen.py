"""Attention over packed sequences (fa_fwd_varlen, fa_fwd_varlen_paged) against a 64-bit
restatement, sequence by sequence, at the tolerances of the other attention calls."""
import math

import pytest
import torch

from exact_io_aware_81_b200 import ops
from oracle import serving
from parity import compare, guarded, guards_intact

pytestmark = pytest.mark.gpu

DEV = "cuda"
SENTINEL = 7.0


def cu(lengths, start=0):
    return torch.tensor([start] + list(lengths), dtype=torch.int64).cumsum(0).to(torch.int32)


def make(nq, nk, Hq, Hkv, d, seed, pad_q=0, pad_k=0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(sum(nq) + pad_q, Hq, d, generator=g).to(torch.bfloat16)
    k, v = (torch.randn(sum(nk) + pad_k, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
    return q, k, v


def run(q, k, v, cq, ck, causal, window=0, out_dtype=torch.bfloat16, scale=None):
    Tq, Hq, d = q.shape
    obuf, o = guarded((Tq, Hq, d), out_dtype, DEV)
    lbuf, lse = guarded((Hq, Tq), torch.float32, DEV)
    o.fill_(SENTINEL)
    lse.fill_(SENTINEL)
    ws = torch.full((ops.varlen_workspace_size(cq.numel() - 1, Tq, Hq, k.shape[1]),), 0xFF, dtype=torch.uint8, device=DEV)
    ops.fwd_varlen(q.to(DEV), k.to(DEV), v.to(DEV), cq.to(DEV), ck.to(DEV) if ck is not None else None, causal=causal,
                   window=window, out_dtype=out_dtype, scale=scale, workspace=ws, out=o, lse=lse)
    status = ops.get_error()
    assert guards_intact(obuf) and guards_intact(lbuf), "write outside the output tensors"
    return o, lse, status


def verify(o, lse, q, k, v, cq, ck, causal, window=0, what="", scale=None):
    scale = scale or 1.0 / math.sqrt(q.shape[2])
    ck = cq if ck is None else ck
    ro, rl = serving.attention_packed(q, k, v, cq, ck, scale, causal, window)
    mine = torch.zeros(q.shape[0], dtype=torch.bool)
    for b in range(cq.numel() - 1):
        mine[int(cq[b]):int(cq[b + 1])] = True
    if mine.any():
        compare(o.cpu()[mine], lse.cpu()[:, mine], ro[mine], rl[:, mine], what)
    assert (o.cpu()[~mine].float() == SENTINEL).all() and (lse.cpu()[:, ~mine] == SENTINEL).all(), "rows of no sequence were written"


LENGTHS = [
    [1],
    [128],
    [5, 1, 64, 130, 1, 300],
    [0, 17, 0, 0, 256, 1, 0],
    [129, 127, 128, 255, 257, 3],
    [700, 1, 2, 400],
]
HEADS = [(4, 2, 128), (8, 8, 64), (6, 2, 64), (8, 1, 128), (3, 1, 128), (2, 2, 128), (32, 1, 64), (40, 1, 128), (10, 2, 64)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda x: "-".join(map(str, x)))
def test_packed_self_attention(lengths, Hq, Hkv, d, causal):
    q, k, v = make(lengths, lengths, Hq, Hkv, d, 1 + len(lengths))
    o, lse, status = run(q, k, v, cu(lengths), None, causal)
    assert status == ops.FA_OK
    verify(o, lse, q, k, v, cu(lengths), None, causal, what=f"{lengths}")


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (3, 1, 64)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 40), (True, 128), (True, 300), (True, 2080), (True, 2 ** 31 - 1), (False, 0)])
def test_other_keys_than_queries(Hq, Hkv, d, causal, window):
    """More keys than queries (chunks), fewer (rows that see nothing), none at all."""
    nq = [1, 200, 130, 300, 5, 64, 0, 260, 3]
    nk = [513, 456, 130, 140, 0, 1, 9, 129, 700]
    q, k, v = make(nq, nk, Hq, Hkv, d, 5, pad_q=9, pad_k=4)
    o, lse, status = run(q, k, v, cu(nq), cu(nk), causal, window)
    assert status == ops.FA_OK
    verify(o, lse, q, k, v, cu(nq), cu(nk), causal, window, f"window {window}")
    if causal:  # 300 queries of 140 keys: the first 160 rows see none
        at = sum(nq[:3])
        assert (o[at:at + 160] == 0).all() and (lse[:, at:at + 160] == -math.inf).all()
    at = sum(nq[:4])
    assert (o[at:at + 5] == 0).all() and (lse[:, at:at + 5] == -math.inf).all()


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (3, 1, 64)])
def test_fp32_output_and_scale(Hq, Hkv, d):
    nq = [33, 1, 257]
    q, k, v = make(nq, nq, Hq, Hkv, d, 6)
    o, lse, status = run(q, k, v, cu(nq), None, True, out_dtype=torch.float32, scale=0.2)
    assert status == ops.FA_OK and o.dtype == torch.float32
    verify(o, lse, q, k, v, cu(nq), None, True, scale=0.2)


@pytest.mark.parametrize("Hq,Hkv,d,window,N", [(8, 2, 128, 0, 320), (3, 1, 64, 0, 336), (4, 4, 128, 0, 512), (8, 2, 128, 200, 320)])
def test_equal_lengths_are_the_dense_call(Hq, Hkv, d, window, N):
    """B sequences of one length: the (B, N, H, d) call, bit for bit, where the tokens fill whole
    pairs of tiles (the tokens left over in one tile take its key tiles in two sums)."""
    B = 3
    q, k, v = make([N] * B, [N] * B, Hq, Hkv, d, 7)
    o, lse, _ = run(q, k, v, cu([N] * B), None, True, window)
    sh = lambda t: t.to(DEV).view(B, N, *t.shape[1:])  # noqa: E731
    od, ld = ops.fwd_bshd(sh(q), sh(k), sh(v), causal=True, window=window)
    assert torch.equal(o.view(B, N, Hq, d), od) and torch.equal(lse.view(Hq, B, N).transpose(0, 1), ld)


def test_slices_of_one_projection():
    n, Hq, Hkv, d = [70, 200, 3], 8, 2, 128
    T = sum(n)
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    dev = qkv.to(DEV)
    parts = (slice(0, Hq), slice(Hq, Hq + Hkv), slice(Hq + Hkv, None))
    o, lse = ops.fwd_varlen(*[dev[:, p] for p in parts], cu(n).to(DEV), causal=True)
    oc, lc = ops.fwd_varlen(*[dev[:, p].contiguous() for p in parts], cu(n).to(DEV), causal=True)
    assert ops.get_error() == ops.FA_OK
    assert torch.equal(o, oc) and torch.equal(lse, lc)
    verify(o, lse, *[qkv[:, p] for p in parts], cu(n), None, True)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (3, 1, 64)])
def test_one_sequence_cannot_reach_another(Hq, Hkv, d, causal, bad):
    """Every odd sequence, and the padding behind the last, holds NaN or infinities."""
    n = [37, 50, 128, 129, 1, 7, 260, 90]
    q, k, v = make(n, n, Hq, Hkv, d, 9, pad_q=40, pad_k=40)
    o0, l0, _ = run(q, k, v, cu(n), None, causal)
    c = cu(n)
    keep = torch.ones(q.shape[0], dtype=torch.bool)
    for b in range(1, len(n), 2):
        keep[int(c[b]):int(c[b + 1])] = False
    keep[int(c[-1]):] = False
    for t in (q, k, v):
        t[~keep] = bad
    o1, l1, status = run(q, k, v, cu(n), None, causal)
    assert status == ops.FA_OK
    assert torch.equal(o0.cpu()[keep], o1.cpu()[keep]) and torch.equal(l0.cpu()[:, keep], l1.cpu()[:, keep])


def test_keys_that_are_not_finite_in_masked_places():
    """A key of the future that is NaN or infinite is masked before it counts."""
    n, Hq, Hkv, d = [100], 4, 2, 128
    q, k, v = make(n, n, Hq, Hkv, d, 10)
    k[60:70] = math.nan
    k[80] = math.inf
    o, lse, _ = run(q, k, v, cu(n), None, True)
    ro, rl = serving.attention_packed(q[:60], k[:60], v[:60], cu([60]), cu([60]), d ** -0.5, True)
    compare(o[:60], lse[:, :60], ro, rl, "rows before the first NaN")


def test_many_sequences_and_a_long_one():
    g = torch.Generator().manual_seed(11)
    n = torch.randint(0, 40, (1500,), generator=g).tolist()
    n[700] = 3001
    Hq, Hkv, d = 4, 1, 64
    q, k, v = make(n, n, Hq, Hkv, d, 12)
    o, lse, status = run(q, k, v, cu(n), None, True)
    assert status == ops.FA_OK
    verify(o, lse, q, k, v, cu(n), None, True)


def test_more_units_than_ctas_repeated():
    """Many units per CTA, drawn in another order each time: the same bits every time."""
    n = [1000, 300, 20, 5, 640, 128, 129, 2000, 77]
    q, k, v = make(n, n, 16, 4, 128, 13)
    o, lse, status = run(q, k, v, cu(n), None, True)
    assert status == ops.FA_OK
    verify(o, lse, q, k, v, cu(n), None, True)
    for _ in range(3):
        o2, l2, _ = run(q, k, v, cu(n), None, True)
        assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_lengths_out_of_range_are_reported():
    """cu_seqlens that descend, or pass the tensors' end: forced into them, and reported; the
    sequences that are in order come out right."""
    n = [50, 60, 70]
    q, k, v = make(n, n, 4, 2, 64, 14)
    good, lse_good, _ = run(q, k, v, cu(n), None, True)
    for c in ([0, 50, 110, 181], [0, 50, 40, 180], [-3, 50, 110, 180], [0, 50, 2 ** 31 - 1, 180], [0, 180, 0, 180]):
        o, lse, status = run(q, k, v, torch.tensor(c, dtype=torch.int32), None, True)
        assert status == ops.FA_ERR_DEVICE_ARG
        if c[:2] == [0, 50]:  # [0, 50, 40, 180] gives rows 40 .. 49 to two sequences
            assert torch.equal(o[:40], good[:40]) and torch.equal(lse[:, :40], lse_good[:, :40])
    o, lse, status = run(q, k, v, cu(n), None, True)
    assert status == ops.FA_OK and torch.equal(o, good)


def test_no_keys_and_no_rows():
    q = torch.randn(5, 4, 64, device=DEV).to(torch.bfloat16)
    none = torch.empty(0, 2, 64, device=DEV, dtype=torch.bfloat16)
    o, lse = ops.fwd_varlen(q, none, none, cu([2, 3]).to(DEV), cu([0, 0]).to(DEV))
    assert ops.get_error() == ops.FA_OK and (o == 0).all() and (lse == -math.inf).all()
    o, lse = ops.fwd_varlen(q[:0], none, none, cu([0, 0]).to(DEV))
    assert tuple(o.shape) == (0, 4, 64) and tuple(lse.shape) == (4, 0)


# ------------------------------------------------------------------------------- pages

def make_paged(nq, nk, Hq, Hkv, d, ps, seed, bad=math.nan):
    """A pool whose unused rows and pages hold NaN."""
    g = torch.Generator().manual_seed(seed)
    q, k, v = make(nq, nk, Hq, Hkv, d, seed)
    need = [-(-n // ps) for n in nk]
    total = sum(need) + 2
    perm = torch.randperm(total, generator=g)
    table = torch.full((len(nk), max(1, max(need))), -1, dtype=torch.int32)
    pools = [torch.full((total, Hkv, ps, d), bad, dtype=torch.bfloat16) for _ in range(2)]
    at = row = 0
    for b, n in enumerate(nk):
        for j in range(need[b]):
            pg = int(perm[at])
            at += 1
            table[b, j] = pg
            m = min(ps, n - j * ps)
            for pool, x in zip(pools, (k, v)):
                pool[pg, :, :m] = x[row + j * ps:row + j * ps + m].transpose(0, 1)
        row += n
    return q, k, v, pools, table


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 100), (False, 0)])
@pytest.mark.parametrize("Hq,Hkv,d", [(4, 2, 128), (8, 8, 64), (6, 2, 128)])
@pytest.mark.parametrize("ps", [16, 48, 64, 128, 384])
def test_paged(ps, Hq, Hkv, d, causal, window):
    nq = [1, 100, 0, 130, 257, 64, 3]
    nk = [300, 163, 20, 130, 900, 64, 0]
    q, k, v, pools, table = make_paged(nq, nk, Hq, Hkv, d, ps, 20 + ps)
    T = sum(nq)
    o = torch.full((T, Hq, d), SENTINEL, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((Hq, T), SENTINEL, device=DEV)
    ops.fwd_varlen_paged(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), table.to(DEV), cu(nq).to(DEV),
                         torch.tensor(nk, dtype=torch.int32).to(DEV), causal=causal, window=window, out=o, lse=lse)
    assert ops.get_error() == ops.FA_OK
    verify(o, lse, q, k, v, cu(nq), cu(nk), causal, window, f"pages of {ps}")
    op, lp, _ = run(q, k, v, cu(nq), cu(nk), causal, window)
    assert torch.equal(o, op) and torch.equal(lse, lp)   # the packed call on the same keys


def test_paged_reports_bad_pages_and_lengths():
    nq, nk, ps = [40, 40, 40], [140, 200, 90], 16
    q, k, v, pools, table = make_paged(nq, nk, 4, 2, 64, ps, 31, bad=0.0)
    dev = [t.to(DEV) for t in (q, pools[0], pools[1])]
    sl = torch.tensor(nk, dtype=torch.int32)
    good, lg = ops.fwd_varlen_paged(*dev, table.to(DEV), cu(nq).to(DEV), sl.to(DEV))
    for bad_page in (-1, pools[0].shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[1, 3] = bad_page
        o, lse = ops.fwd_varlen_paged(*dev, t.to(DEV), cu(nq).to(DEV), sl.to(DEV))
        assert ops.get_error() == ops.FA_ERR_DEVICE_ARG
        assert torch.equal(o[:40], good[:40]) and torch.equal(o[80:], good[80:])
        k2, v2 = k.clone(), v.clone()   # its keys and values read as zeros
        k2[140 + 48:140 + 64] = 0
        v2[140 + 48:140 + 64] = 0
        ro, rl = serving.attention_packed(q, k2, v2, cu(nq), cu(nk), 64 ** -0.5, True)
        compare(o, lse, ro, rl, "zero page")
    for length in (-1, ps * table.shape[1] + 1):
        s = sl.clone()
        s[2] = length
        o, lse = ops.fwd_varlen_paged(*dev, table.to(DEV), cu(nq).to(DEV), s.to(DEV))
        assert ops.get_error() == ops.FA_ERR_DEVICE_ARG
        assert torch.equal(o[:80], good[:80])


# ---------------------------------------------------------------- streams and graphs

def test_two_streams_with_their_own_workspaces():
    n = [400, 129, 800, 33]
    q, k, v = (t.to(DEV) for t in make(n, n, 8, 2, 128, 40))
    c = cu(n).to(DEV)
    want, wl = ops.fwd_varlen(q, k, v, c, causal=True)
    full, fl = ops.fwd_varlen(q, k, v, c, causal=False)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    ws = [torch.empty(ops.varlen_workspace_size(len(n), sum(n), 8, 2), dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for _ in range(5):
        outs.append((ops.fwd_varlen(q, k, v, c, causal=True, workspace=ws[0], stream=a), want, wl))
        outs.append((ops.fwd_varlen(q, k, v, c, causal=False, workspace=ws[1], stream=b), full, fl))
    torch.cuda.synchronize()
    for (o, l), wo, w in outs:
        assert torch.equal(o, wo) and torch.equal(l, w)


@pytest.mark.parametrize("paged", [False, True])
def test_own_workspace_on_another_stream(paged):
    """A call that makes its workspace itself, on a stream that is still busy: what the current
    stream allocates and writes after the call returned must not be that workspace."""
    n, ps = [400, 129, 800, 33] * 8, 64
    q, k, v = (t.to(DEV) for t in make(n, n, 8, 2, 128, 43))
    c = cu(n).to(DEV)
    if paged:
        mp = 16
        table = torch.arange(len(n) * mp, dtype=torch.int32, device=DEV).view(len(n), mp)
        kp, vp = (torch.randn(len(n) * mp, 2, ps, 128, device=DEV).to(torch.bfloat16) for _ in range(2))
        lens = torch.tensor(n, dtype=torch.int32, device=DEV)
    call = lambda **kw: (ops.fwd_varlen_paged(q, kp, vp, table, c, lens, **kw) if paged else
                         ops.fwd_varlen(q, k, v, c, causal=True, **kw))
    want, wl = call()
    o, lse = torch.empty_like(want), torch.empty_like(wl)
    size = ops.varlen_workspace_size(len(n), sum(n), 8, 2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms
    call(out=o, lse=lse, stream=side)
    fill = [torch.full((size,), 0x11, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert ops.get_error() == ops.FA_OK and len(fill) == 4
    assert torch.equal(o, want) and torch.equal(lse, wl)


def test_captured_and_replayed_with_other_lengths():
    """The lengths are read on the device: a replay serves whatever the buffers hold then."""
    Hq, Hkv, d, T = 8, 2, 128, 600
    q, k, v = (t.to(DEV) for t in make([T], [T], Hq, Hkv, d, 41))
    c = cu([100, 200, 300]).to(DEV)
    ws = torch.empty(ops.varlen_workspace_size(3, T, Hq, Hkv), dtype=torch.uint8, device=DEV)
    o, lse = torch.empty_like(q), torch.empty(Hq, T, device=DEV)
    ops.fwd_varlen(q, k, v, c, causal=True, workspace=ws, out=o, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.fwd_varlen(q, k, v, c, causal=True, workspace=ws, out=o, lse=lse)
    for n in ([100, 200, 300], [1, 598, 1], [0, 0, 600], [300, 0, 299]):
        c.copy_(cu(n))
        want, wl = ops.fwd_varlen(q, k, v, c, causal=True)
        ws.fill_(0x77)
        graph.replay()
        torch.cuda.synchronize()
        m = sum(n)
        assert torch.equal(o[:m], want[:m]) and torch.equal(lse[:, :m], wl[:, :m])


def test_long_packed_offsets():
    """A packed q of more than 2^31 elements: the last sequence lies beyond 32-bit offsets."""
    Hq, Hkv, d = 32, 1, 128
    T = (1 << 19) + 4096 + 37   # T * Hq * d > 2^31
    q = torch.zeros(T, Hq, d, device=DEV, dtype=torch.bfloat16)
    k, v = (torch.zeros(T, Hkv, d, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    n = 37 + 100
    g = torch.Generator().manual_seed(42)
    qs, ks, vs = (torch.randn(n, h, d, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    q[T - n:], k[T - n:], v[T - n:] = qs.to(DEV), ks.to(DEV), vs.to(DEV)
    c = torch.tensor([T - n, T], dtype=torch.int32)  # the rows before belong to nobody
    o, lse = ops.fwd_varlen(q, k, v, c.to(DEV), causal=True)
    assert ops.get_error() == ops.FA_OK
    ro, rl = serving.attention(qs, ks, vs, d ** -0.5, True)
    compare(o[T - n:], lse[:, T - n:], ro, rl, "far rows")


def test_refusals():
    q = torch.zeros(4, 4, 64, device=DEV, dtype=torch.bfloat16)
    k = torch.zeros(4, 2, 64, device=DEV, dtype=torch.bfloat16)
    c = cu([4]).to(DEV)
    bad = [lambda: ops.fwd_varlen(q.float(), k, k, c), lambda: ops.fwd_varlen(q, k, k[:3], c),
           lambda: ops.fwd_varlen(q, k, k, c.long()), lambda: ops.fwd_varlen(q, k, k, c[:1]),
           lambda: ops.fwd_varlen(q.transpose(0, 1), k, k, c), lambda: ops.fwd_varlen(q, k, k, c, out_dtype=torch.float16),
           lambda: ops.fwd_varlen(q, k, k, c, out=torch.empty(4, 4, 32, device=DEV, dtype=torch.bfloat16)),
           lambda: ops.fwd_varlen(q, k, k, c.cpu())]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    def status(f):
        with pytest.raises(ops.FAError) as e:
            f()
        return e.value.status
    assert status(lambda: ops.fwd_varlen(q, k, k, c, window=4)) == ops.FA_ERR_INVALID      # needs causal
    assert status(lambda: ops.fwd_varlen(q, k, k, c, causal=True, window=-1)) == ops.FA_ERR_INVALID
    assert status(lambda: ops.fwd_varlen(q, k, k, c, scale=0.0)) == ops.FA_ERR_INVALID
    small = torch.empty(16, device=DEV, dtype=torch.uint8)
    assert status(lambda: ops.fwd_varlen(q, k, k, c, workspace=small)) == ops.FA_ERR_WORKSPACE


@pytest.mark.parametrize("Hq,Hkv,d", [(4, 4, 128), (8, 2, 64), (3, 1, 128)])
@pytest.mark.parametrize("B", [1, 31, 33, 70])
def test_one_wave_of_units(B, Hq, Hkv, d):
    """Few enough units for a CTA each: no plan is made, every CTA finds its own job -- among
    sequences of no tokens, in every step of 32 sequences, and past the last job."""
    g = torch.Generator().manual_seed(B)
    n = [0] * B
    for b in {0, B // 2, B - 1}:
        n[b] = int(torch.randint(1, 60, (1,), generator=g))
    n[B // 2] = 0 if B > 2 else n[B // 2]
    if B > 32:
        n[32] = 9
    nk = [x + int(torch.randint(0, 700, (1,), generator=g)) for x in n]
    q, k, v = make(n, nk, Hq, Hkv, d, 50 + B, pad_q=3, pad_k=2)
    o, lse, status = run(q, k, v, cu(n), cu(nk), True)
    assert status == ops.FA_OK
    verify(o, lse, q, k, v, cu(n), cu(nk), True)
    bad = cu(n)
    bad[-1] = q.shape[0] + 1
    assert run(q, k, v, bad, cu(nk), True)[2] == ops.FA_ERR_DEVICE_ARG
