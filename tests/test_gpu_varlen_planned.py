"""Packed attention by the kernels that follow a plan: calls of more units than the GPU has SMs.

Such a call runs the plan kernel and then one of two variants of the attention kernel, SHORT for a
few tokens per sequence against long contexts in few units, LONG otherwise; a call of fewer units runs SHORT
without a plan (WAVE).  Every test here states the variant it is about and checks that its sizes
choose it: the rule is restated below, and a call leaves its plan in the workspace.  All outputs are
compared with the 64-bit restatement at the tolerances of the other attention calls."""
import math
import re

import pytest
import torch

from exact_io_aware_81_b200 import ops
from oracle import serving
from parity import compare, guarded, guards_intact
from test_gpu_varlen import SENTINEL, cu, make, make_paged, verify

pytestmark = pytest.mark.gpu

DEV = "cuda"
WAVE, SHORT, LONG = "wave", "short", "long"


def pack_of(R):
    return next(p for p in range(min(R, 32), 0, -1) if R % p == 0)


def variant_of(B, Tq, Hq, Hkv, all_keys):
    """The kernel that a call gets (all_keys: rows of k, or what the pages or the table can hold)."""
    pack = pack_of(Hq // Hkv)
    tokens = 128 // pack
    bound = (Tq // (2 * tokens) + B) * (Hq // pack)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if bound <= sms:
        return WAVE
    return SHORT if Tq <= 4 * B * tokens and all_keys >= 1024 * B and bound <= 5 * sms else LONG


def units_of(nq, Hq, Hkv):
    pack = pack_of(Hq // Hkv)
    return sum(-(-n // (2 * (128 // pack))) for n in nq) * (Hq // pack)


def call(q, k, v, cq, ck, causal, window=0, out_dtype=torch.bfloat16, paged=None, ws=None):
    """-> (o, lse, status, jobs of the plan or None); `paged`: (pools, table, lengths)."""
    Tq, Hq, d = q.shape
    obuf, o = guarded((Tq, Hq, d), out_dtype, DEV)
    lbuf, lse = guarded((Hq, Tq), torch.float32, DEV)
    o.fill_(SENTINEL)
    lse.fill_(SENTINEL)
    Hkv = k.shape[1]
    ws = torch.full((ops.varlen_workspace_size(cq.numel() - 1, Tq, Hq, Hkv),), 0xFF, dtype=torch.uint8, device=DEV)
    kw = dict(causal=causal, window=window, out_dtype=out_dtype, workspace=ws, out=o, lse=lse)
    if paged:
        pools, table, lens = paged
        ops.fwd_varlen_paged(q.to(DEV), pools[0].to(DEV), pools[1].to(DEV), table.to(DEV), cq.to(DEV), lens.to(DEV), **kw)
    else:
        ops.fwd_varlen(q.to(DEV), k.to(DEV), v.to(DEV), cq.to(DEV), ck.to(DEV), **kw)
    status = ops.get_error()
    assert guards_intact(obuf) and guards_intact(lbuf), "write outside the output tensors"
    jobs = int(ws[:4].view(torch.int32))
    return o, lse, status, None if jobs == -1 else jobs


def lengths(kind, B, seed, most):
    """Query and key counts: SHORT over contexts of 1024 keys and more on average (some of none, and
    some shorter than their queries), LONG over those of self-attention and less."""
    g = torch.Generator().manual_seed(seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    nq = [r(1, most) for _ in range(B)]
    if kind == SHORT:
        nk = [n + r(900, 1700) for n in nq]
        nk[1], nk[2], nk[3], nk[4] = 0, 5, nq[3] + 120, nq[4] + 128   # none, fewer, one tile, two
        nk[5] += 3000
        nk[6] += 1200
    else:
        nk = [max(0, n + r(-60, 200)) for n in nq]
        nk[1] = 0
    nq[B // 2] = 0
    return nq, nk


# (kind, B, most tokens, Hq, Hkv, d): units per CTA from just over one on, every pack form
CASES = [
    (SHORT, 45, 90, 4, 4, 64),      # 180 units: numbers drawn late
    (SHORT, 45, 300, 4, 4, 128),    # pairs of tiles beside twins
    (SHORT, 80, 70, 8, 2, 128),
    (SHORT, 160, 30, 3, 1, 64),     # 126 rows a tile
    (SHORT, 39, 90, 16, 16, 64),    # 608 units: more than four a CTA, numbers drawn early
    (SHORT, 39, 40, 16, 16, 128),
    (LONG, 20, 300, 16, 16, 64),
    (LONG, 20, 300, 16, 16, 128),
    (LONG, 60, 200, 12, 4, 64),     # 126 rows a tile
    (LONG, 50, 200, 16, 4, 128),
    (LONG, 150, 9, 32, 1, 128),     # four tokens a tile
]
IDS = [f"{c[0]}-{c[3]}x{c[4]}x{c[5]}-{c[2]}" for c in CASES]


def build(case, seed=1):
    kind, B, most, Hq, Hkv, d = case
    nq, nk = lengths(kind, B, seed, most)
    assert units_of(nq, Hq, Hkv) > torch.cuda.get_device_properties(0).multi_processor_count
    return nq, nk, Hq, Hkv, d


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 130), (True, 700), (False, 0)])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_planned(case, causal, window):
    nq, nk, Hq, Hkv, d = build(case)
    q, k, v = make(nq, nk, Hq, Hkv, d, 60, pad_q=5, pad_k=7)
    assert variant_of(len(nq), q.shape[0], Hq, Hkv, k.shape[0]) == case[0]
    o, lse, status, jobs = call(q, k, v, cu(nq), cu(nk), causal, window)
    assert status == ops.FA_OK and jobs == units_of(nq, Hq, Hkv) // (Hq // pack_of(Hq // Hkv))
    verify(o, lse, q, k, v, cu(nq), cu(nk), causal, window, f"{case} window {window}")


@pytest.mark.parametrize("window", [0, 130])
@pytest.mark.parametrize("case", [c for c in CASES if c[3] != 3], ids=[i for i, c in zip(IDS, CASES) if c[3] != 3])
def test_planned_fp32_output(case, window):
    nq, nk, Hq, Hkv, d = build(case, 2)
    q, k, v = make(nq, nk, Hq, Hkv, d, 61)
    assert variant_of(len(nq), q.shape[0], Hq, Hkv, k.shape[0]) == case[0]
    o, lse, status, jobs = call(q, k, v, cu(nq), cu(nk), True, window, out_dtype=torch.float32)
    assert status == ops.FA_OK and jobs and o.dtype == torch.float32
    verify(o, lse, q, k, v, cu(nq), cu(nk), True, window)


@pytest.mark.parametrize("causal,window,out_dtype", [(True, 0, torch.bfloat16), (True, 150, torch.bfloat16),
                                                     (False, 0, torch.bfloat16), (True, 0, torch.float32),
                                                     (True, 150, torch.float32)])
@pytest.mark.parametrize("ps", [16, 48, 128, 384])
@pytest.mark.parametrize("case", [CASES[0], CASES[2], CASES[5], CASES[6], CASES[9]], ids=lambda c: f"{c[0]}-{c[3]}x{c[4]}x{c[5]}")
def test_planned_paged(case, ps, causal, window, out_dtype):
    """Pools whose unused rows and pages hold NaN; the pages are few enough for LONG to be chosen."""
    nq, nk, Hq, Hkv, d = build(case, 3)
    q, k, v, pools, table = make_paged(nq, nk, Hq, Hkv, d, ps, 62 + ps)
    cap = ps * min(pools[0].shape[0], table.numel())
    assert variant_of(len(nq), q.shape[0], Hq, Hkv, cap) == case[0]
    o, lse, status, jobs = call(q, k, v, cu(nq), None, causal, window, out_dtype,
                                paged=(pools, table, torch.tensor(nk, dtype=torch.int32)))
    assert status == ops.FA_OK and jobs
    verify(o, lse, q, k, v, cu(nq), cu(nk), causal, window, f"{case} pages of {ps}")


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", [CASES[0], CASES[2], CASES[4], CASES[6], CASES[8], CASES[9]],
                         ids=lambda c: f"{c[0]}-{c[3]}x{c[4]}x{c[5]}")
def test_planned_isolation(case, causal, bad):
    """Every odd sequence, and the padding behind the last, holds NaN or infinities: the others keep
    their bits."""
    nq, nk, Hq, Hkv, d = build(case, 4)
    q, k, v = make(nq, nk, Hq, Hkv, d, 63, pad_q=20, pad_k=20)
    cq, ck = cu(nq), cu(nk)
    assert variant_of(len(nq), q.shape[0], Hq, Hkv, k.shape[0]) == case[0]
    o0, l0, _, _ = call(q, k, v, cq, ck, causal)
    rows, keys = torch.ones(q.shape[0], dtype=torch.bool), torch.ones(k.shape[0], dtype=torch.bool)
    for b in range(1, len(nq), 2):
        rows[int(cq[b]):int(cq[b + 1])] = False
        keys[int(ck[b]):int(ck[b + 1])] = False
    rows[int(cq[-1]):] = False
    keys[int(ck[-1]):] = False
    q[~rows] = bad
    k[~keys] = bad
    v[~keys] = bad
    o1, l1, status, jobs = call(q, k, v, cq, ck, causal)
    assert status == ops.FA_OK and jobs
    assert torch.equal(o0.cpu()[rows], o1.cpu()[rows]) and torch.equal(l0.cpu()[:, rows], l1.cpu()[:, rows])


@pytest.mark.parametrize("case", [CASES[0], CASES[2], CASES[4], CASES[6], CASES[9]], ids=lambda c: f"{c[0]}-{c[3]}x{c[4]}x{c[5]}")
def test_planned_repeats_its_bits(case):
    """Units are drawn in another order each time; the outputs are the same bits."""
    nq, nk, Hq, Hkv, d = build(case, 5)
    q, k, v = (t.to(DEV) for t in make(nq, nk, Hq, Hkv, d, 64))
    cq, ck = cu(nq).to(DEV), cu(nk).to(DEV)
    o, lse = ops.fwd_varlen(q, k, v, cq, ck, causal=True)
    for _ in range(20):
        o2, l2 = ops.fwd_varlen(q, k, v, cq, ck, causal=True)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    assert ops.get_error() == ops.FA_OK


@pytest.mark.parametrize("case", [CASES[0], CASES[4], CASES[6]], ids=lambda c: f"{c[0]}-{c[3]}x{c[4]}x{c[5]}")
def test_planned_lengths_out_of_range(case):
    """cu_seqlens that descend or pass the ends are forced into the tensors and reported, by the plan
    kernel as by the planless one; the sequences before the first bad one come out right."""
    nq, nk, Hq, Hkv, d = build(case, 6)
    q, k, v = make(nq, nk, Hq, Hkv, d, 65)
    cq, ck = cu(nq), cu(nk)
    good, lg, status, _ = call(q, k, v, cq, ck, True)
    assert status == ops.FA_OK
    B, T = len(nq), q.shape[0]
    at = int(cq[10])
    for change in ((10, at - 1, -1), (B, T + 1, B - 1), (0, -3, None), (B, 2 ** 31 - 1, B - 1), (20, 0, 19)):
        i, value, until = change
        bad = cq.clone()
        bad[i] = value
        if i == 10:
            bad[11:] = bad[11:].flip(0)   # a long descent
        o, lse, status, jobs = call(q, k, v, bad, ck, True)
        assert status == ops.FA_ERR_DEVICE_ARG and jobs is not None
        if until and until > 0 and until == B - 1:
            n = int(cq[until])
            assert torch.equal(o[:n], good[:n]) and torch.equal(lse[:, :n], lg[:, :n])
    # every second sequence all tokens: more jobs than the plan holds
    bad = torch.zeros(B + 1, dtype=torch.int32)
    bad[1::2] = T
    _, _, status, jobs = call(q, k, v, bad, ck, True)
    pack = pack_of(Hq // Hkv)
    assert status == ops.FA_ERR_DEVICE_ARG and jobs <= T // (2 * (128 // pack)) + B
    bad_k = ck.clone()
    bad_k[B] = k.shape[0] + 1
    assert call(q, k, v, cq, bad_k, True)[2] == ops.FA_ERR_DEVICE_ARG
    o, lse, status, _ = call(q, k, v, cq, ck, True)
    assert status == ops.FA_OK and torch.equal(o, good)


@pytest.mark.parametrize("case", [CASES[0], CASES[4], CASES[6]], ids=lambda c: f"{c[0]}-{c[3]}x{c[4]}x{c[5]}")
def test_planned_captured_and_replayed(case):
    """A replay makes its plan again, from what the lengths' buffers hold then."""
    nq, nk, Hq, Hkv, d = build(case, 7)
    q, k, v = (t.to(DEV) for t in make(nq, nk, Hq, Hkv, d, 66))
    cq, ck = cu(nq).to(DEV), cu(nk).to(DEV)
    B, T = len(nq), q.shape[0]
    ws = torch.empty(ops.varlen_workspace_size(B, T, Hq, Hkv), dtype=torch.uint8, device=DEV)
    o, lse = torch.empty_like(q), torch.empty(Hq, T, device=DEV)
    run = lambda **kw: ops.fwd_varlen(q, k, v, cq, ck, causal=True, **kw)  # noqa: E731
    run(workspace=ws, out=o, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(workspace=ws, out=o, lse=lse)
    for swap in (0, 3, 11):
        n2, m2 = nq[swap:] + nq[:swap], nk[swap:] + nk[:swap]
        if swap == 11:
            n2[0] += n2[1]
            n2[1] = 0
        cq.copy_(cu(n2))
        ck.copy_(cu(m2))
        want, wl = run()
        o.fill_(SENTINEL)
        ws.fill_(0x77)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, wl)
    verify(want, wl, q.cpu(), k.cpu(), v.cpu(), cu(n2), cu(m2), True)
    assert ops.get_error() == ops.FA_OK


def test_the_restated_rule_names_the_kernel_that_runs():
    """The names of the launched kernels, from the profiler, against the rule restated above."""
    from torch.profiler import ProfilerActivity, profile
    sizes = [CASES[0], CASES[4], CASES[6], CASES[8], (WAVE, 9, 60, 4, 4, 64)]
    seen = 0
    for case in sizes:
        kind, B, most, Hq, Hkv, d = case
        nq, nk = lengths(SHORT if kind == SHORT else LONG, B, 8, most)
        for window in (0, 50):
            q, k, v = (t.to(DEV) for t in make(nq, nk, Hq, Hkv, d, 67))
            assert variant_of(B, q.shape[0], Hq, Hkv, k.shape[0]) == kind
            cq, ck = cu(nq).to(DEV), cu(nk).to(DEV)
            ops.fwd_varlen(q, k, v, cq, ck, causal=True, window=window)
            torch.cuda.synchronize()
            with profile(activities=[ProfilerActivity.CUDA]) as prof:
                ops.fwd_varlen(q, k, v, cq, ck, causal=True, window=window)
                torch.cuda.synchronize()
            names = [e.key for e in prof.key_averages()]
            args = [re.search(r"fa_varlen_kernel<([^>]*)>", n) for n in names]
            args = [[{"true": 1, "false": 0}.get(x.strip()) if x.strip() in ("true", "false") else int(x)
                     for x in m.group(1).split(",")] for m in args if m]
            if not args:
                continue   # no profiler on this machine
            seen += 1
            assert args == [[d, 0, 1 if window else 0, 0, 0 if kind == LONG else 1]]
            assert any("fa_varlen_plan_kernel" in n for n in names) == (kind != WAVE)
    if not seen:
        pytest.skip("the profiler reports no kernels here")


def test_more_jobs_than_an_int_counts():
    """cu_seqlens that go back to 0 again and again: 2048 sequences of 2^20 jobs each, 2^31 in all.
    The plan stops at what it holds (2^20 + 4096 jobs: the first sequence and a bit of the next),
    and reports.  In 32 bits the sum would wrap, and jobs start at negative rows."""
    Hq, Hkv, d, B, T = 32, 1, 64, 4096, 1 << 23
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 70 GB of device memory")
    q = torch.zeros(T, Hq, d, dtype=torch.bfloat16, device=DEV)
    o = torch.full_like(q, SENTINEL)
    lse = torch.full((Hq, T), SENTINEL, device=DEV)
    v = torch.arange(1, d + 1, device=DEV).to(torch.bfloat16).view(1, 1, d)
    cq = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    cq[1::2] = T
    ck = torch.ones(B + 1, dtype=torch.int32, device=DEV)
    ck[0] = 0   # one key, of the first sequence
    ws = torch.full((ops.varlen_workspace_size(B, T, Hq, Hkv),), 0xFF, dtype=torch.uint8, device=DEV)
    ops.fwd_varlen(q, v, v, cq, ck, workspace=ws, out=o, lse=lse)
    assert ops.get_error() == ops.FA_ERR_DEVICE_ARG
    assert int(ws[:4].view(torch.int32)) == T // 8 + B
    n = 8 * B   # rows that the second whole sequence (without keys) has too
    for a in range(0, T, T // 16):
        part, z = o[a:a + T // 16], lse[:, a:a + T // 16]
        ok, oz = (part == v).all(-1), z == 0
        if a == 0:
            ok[:n] |= (part[:n] == 0).all(-1)
            oz[:, :n] |= z[:, :n] == -math.inf
        assert ok.all() and oz.all()


def test_many_units_are_long_whatever_the_pool_could_hold():
    """512 short prompts whose table and pool could hold 8192 keys each: five units a CTA or more take
    the LONG kernel (157 us where SHORT took 211)."""
    from torch.profiler import ProfilerActivity, profile
    B, nq, Hq, Hkv, d, ps, mp = 512, 64, 8, 2, 64, 64, 128
    T = B * nq
    g = torch.Generator().manual_seed(70)
    q, k, v = make([T], [T], Hq, Hkv, d, 71)
    pool = 17 * B   # 1088 keys a sequence
    kp, vp = (torch.full((pool, Hkv, ps, d), math.nan, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pages = torch.randperm(pool, generator=g)[:B]
    table = torch.full((B, mp), -1, dtype=torch.int32)
    table[:, 0] = pages.to(torch.int32)
    for p, x in ((kp, k), (vp, v)):
        p[pages.to(DEV)] = x.to(DEV).view(B, ps, Hkv, d).transpose(1, 2)
    n = cu([nq] * B)
    assert variant_of(B, T, Hq, Hkv, ps * pool) == LONG
    args = (q.to(DEV), kp, vp, table.to(DEV), n.to(DEV), torch.full((B,), nq, dtype=torch.int32, device=DEV))
    o, lse = ops.fwd_varlen_paged(*args)
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA]) as prof:
        o2, l2 = ops.fwd_varlen_paged(*args)
        torch.cuda.synchronize()
    assert ops.get_error() == ops.FA_OK and torch.equal(o, o2) and torch.equal(lse, l2)
    some = [0, 1, 100, 511]
    for b in some:
        s = slice(b * nq, (b + 1) * nq)
        ro, rl = serving.attention(q[s], k[s], v[s], d ** -0.5, True)
        compare(o[s], lse[:, s], ro, rl, f"sequence {b}")
    names = [m.group(1) for e in prof.key_averages() if (m := re.search(r"fa_varlen_kernel<([^>]*)>", e.key))]
    if names:
        assert len(names) == 1 and names[0].split(",")[-1].strip() in ("false", "0"), names


def test_short_units_cost_what_they_cost():
    """Single tokens on contexts of 4096, SHORT, with just less and just more than four units a CTA
    (where numbers are drawn late and early): a third more units may not take twice the time.  (While
    the producer's look at the next unit's Q slot could suspend it, they took four times as long.)"""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    Hq, Hkv, d, ps, ctx = 32, 8, 128, 64, 4096
    times = {}
    for B in (3 * sms // 8, -(-4 * sms // 8)):
        mp = ctx // ps
        assert variant_of(B, B, Hq, Hkv, B * ctx) == SHORT
        kp, vp = (torch.randn(B * mp, Hkv, ps, d, device=DEV).to(torch.bfloat16) for _ in range(2))
        table = torch.randperm(B * mp, device=DEV).to(torch.int32).view(B, mp)
        q = torch.randn(B, Hq, d, device=DEV).to(torch.bfloat16)
        cq, lens = torch.arange(B + 1, dtype=torch.int32, device=DEV), torch.full((B,), ctx, dtype=torch.int32, device=DEV)
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        best = math.inf
        for _ in range(6):
            a.record()
            o, lse = ops.fwd_varlen_paged(q, kp, vp, table, cq, lens)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        times[B] = best
        od, ld = ops.decode_paged(q, kp, vp, table, lens)
        compare(o.cpu(), lse.cpu(), od.cpu().double(), ld.cpu().double().T, "against the decode kernel")
    assert ops.get_error() == ops.FA_OK
    few, many = times.values()
    assert many < 2 * few, times
