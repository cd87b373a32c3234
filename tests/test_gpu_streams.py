"""Calls with stream= on a stream that is still busy, which make their outputs themselves: what the
current stream allocates and writes after the call returned must not be those outputs, also when
the caller has dropped them by then."""
import numpy as np
import pytest
import torch

from exact_io_aware_81_b200 import ops
from oracle import serving

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).to(DEV)


def randn(*shape, seed=0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def busy_stream():
    """A side stream with some 10 ms of work in front of whatever comes."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    return side


def fill_like(sizes):
    """Blocks of these sizes on the current stream, written now: the allocator would serve them from
    whatever was returned to that stream's pool.  -> a check that they are as written."""
    blocks = [torch.full((n,), 0x11, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(4)]

    def intact():
        torch.cuda.synchronize()
        return all(bool((b == 0x11).all()) for b in blocks)
    return intact


def test_the_copy_list_is_dropped_at_once():
    """Compaction and its copy in one expression: the list of moves has no other owner."""
    S, ps, mp, N, d = 300, 16, 20, 4000, 64
    r = np.random.RandomState(1)
    p = serving.Pages(S, mp, N, ps)
    p.reserve(r.randint(0, 150, S))
    p.free(np.arange(0, S, 3))
    state = i32(p.table), i32(p.lens), i32(p.ref)
    kp, vp = (torch.randint(0, 255, (N, 1, ps, d), dtype=torch.uint8, device=DEV) for _ in range(2))
    wk, wv = kp.clone(), vp.clone()
    busy = busy_stream()
    ops.pages_copy(kp, vp, ops.pages_compact(*state, ps, stream=busy), stream=busy)
    intact = fill_like([8 * (N // 2), ops.pages_compact_workspace_size(N)])
    assert intact() and ops.get_error() == ops.FA_OK
    moves = torch.from_numpy(p.compact()).long()
    moves = moves[moves[:, 0] >= 0].to(DEV)
    assert len(moves) > 100
    wk[moves[:, 1]], wv[moves[:, 1]] = wk[moves[:, 0]], wv[moves[:, 0]]
    assert torch.equal(kp, wk) and torch.equal(vp, wv)


def test_outputs_are_dropped_at_once():
    n, Hq, Hkv, d = [400, 129, 800, 33] * 8, 8, 2, 128
    T = sum(n)
    q, k, v = randn(T, Hq, d), randn(T, Hkv, d, seed=1), randn(T, Hkv, d, seed=2)
    c, pos, inv = i32(np.cumsum([0] + n)), i32(np.arange(T)), torch.ones(64, device=DEV)
    want, wl = ops.fwd_varlen(q, k, v, c, causal=True)
    wq, wk = ops.rope(q, k, pos, inv)
    busy = busy_stream()
    o = ops.fwd_varlen(q, k, v, c, causal=True, stream=busy)[0]      # the LSE has no owner
    lse = ops.fwd_varlen(q, k, v, c, causal=True, stream=busy)[1]    # nor has this O
    qo = ops.rope(q, k, pos, inv, stream=busy)[0]
    ko = ops.rope(q, k, pos, inv, stream=busy)[1]
    intact = fill_like([4 * Hq * T, 2 * T * Hq * d, 2 * T * Hkv * d])
    assert intact() and ops.get_error() == ops.FA_OK
    assert torch.equal(o, want) and torch.equal(lse, wl) and torch.equal(qo, wq) and torch.equal(ko, wk)


def test_outputs_do_not_take_what_the_current_stream_still_uses():
    """The current stream has work queued on blocks that were dropped: a call on another stream that
    makes outputs of that size must not be given them."""
    T, Hq, d = 4096, 8, 128
    q, pos, inv = randn(T, Hq, d, seed=3), i32(np.arange(T)), torch.ones(64, device=DEV)
    side = torch.cuda.Stream()
    want = ops.rope(q, None, pos, inv)[0]
    total = torch.zeros((), device=DEV, dtype=torch.float64)
    torch.cuda.synchronize()
    ones = torch.ones(T, Hq, d, device=DEV, dtype=torch.bfloat16)
    torch.cuda._sleep(20_000_000)
    total += ones.double().sum()
    del ones
    got = ops.rope(q, None, pos, inv, stream=side)[0]   # side does not wait for the current stream
    torch.cuda.synchronize()
    assert float(total) == T * Hq * d
    assert torch.equal(got, want) and ops.get_error() == ops.FA_OK


def test_a_raw_stream_and_the_current_one():
    """Another framework's stream (only a handle), and the current stream named explicitly."""
    T, Hq, d = 100, 4, 64
    q, pos, inv = randn(T, Hq, d, seed=4), i32(np.arange(T)), torch.ones(32, device=DEV)
    want = ops.rope(q, None, pos, inv)[0]
    side = torch.cuda.Stream()

    class Handle:
        cuda_stream = side.cuda_stream

    torch.cuda.synchronize()
    a = ops.rope(q, None, pos, inv, stream=Handle())[0]
    b = ops.rope(q, None, pos, inv, stream=torch.cuda.current_stream())[0]
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want) and ops.get_error() == ops.FA_OK


def test_decode_workspace_and_outputs_on_a_busy_stream():
    """The decode's partial results lie in a workspace that nobody holds once the call has returned."""
    B, Hq, Hkv, N, d = 4, 8, 2, 5000, 128
    q, kc, vc = randn(B, Hq, d), randn(B, Hkv, N, d, seed=1), randn(B, Hkv, N, d, seed=2)
    sl = i32([5000, 1, 3000, 777])
    want, wl = ops.decode(q, kc, vc, sl)
    x, k, v = randn(2, Hq, 600, d, seed=3), randn(2, Hkv, 600, d, seed=4), randn(2, Hkv, 600, d, seed=5)
    wx, wxl = ops.fwd(x, k, v, causal=True)
    busy = busy_stream()
    o = ops.decode(q, kc, vc, sl, stream=busy)[0]
    lse = ops.decode(q, kc, vc, sl, stream=busy)[1]
    xo = ops.fwd(x, k, v, causal=True, stream=busy)[0]
    xl = ops.fwd(x, k, v, causal=True, stream=busy)[1]
    intact = fill_like([ops.decode_workspace_size(B, Hq, N, d), 2 * B * Hq * d, 4 * B * Hq, wx.numel() * 2, wxl.numel() * 4])
    assert intact() and ops.get_error() == ops.FA_OK
    assert torch.equal(o, want) and torch.equal(lse, wl) and torch.equal(xo, wx) and torch.equal(xl, wxl)


def test_captured_on_a_forked_stream():
    """Inside a capture: a side stream that joined it runs calls that make their outputs and their
    workspace, some dropped at once."""
    n, Hq, Hkv, d = [400, 129, 800, 33] * 8, 8, 2, 128
    T = sum(n)
    q, k, v = randn(T, Hq, d), randn(T, Hkv, d, seed=1), randn(T, Hkv, d, seed=2)
    c, pos, inv = i32(np.cumsum([0] + n)), i32(np.arange(T)), torch.ones(64, device=DEV)
    side = torch.cuda.Stream()
    want, wl = ops.fwd_varlen(q, k, v, c, causal=True)
    wq, wk = ops.rope(q, k, pos, inv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        o = ops.fwd_varlen(q, k, v, c, causal=True, stream=side)[0]
        lse = ops.fwd_varlen(q, k, v, c, causal=True, stream=side)[1]
        qo, ko = ops.rope(q, k, pos, inv)
        here.wait_stream(side)
    for _ in range(3):
        for t in (o, lse, qo, ko):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(lse, wl) and torch.equal(qo, wq) and torch.equal(ko, wk)
    assert ops.get_error() == ops.FA_OK


def planned_calls():
    """Calls of more units than CTAs, both variants, each with a workspace of its own, and their results
    one at a time: -> [(call(stream), wanted)]."""
    Hq, Hkv, d, ps = 16, 8, 64, 64
    calls = []
    for seed, (B, most, ctx) in enumerate(((24, 60, 1500), (30, 300, 0), (28, 90, 1100), (40, 200, 60))):
        r = np.random.RandomState(seed)
        nq, cached = r.randint(1, most + 1, B), r.randint(0, 2 * ctx + 1, B) if ctx else np.zeros(B, int)
        nk = nq + cached
        T, need = int(nq.sum()), -(-nk // ps)
        table = np.full((B, int(need.max())), -1, np.int32)
        perm, at = r.permutation(int(need.sum())), 0
        for b, m in enumerate(need):
            table[b, :m] = perm[at:at + m]
            at += m
        q, kp, vp = randn(T, Hq, d, seed=seed), randn(at, Hkv, ps, d, seed=seed + 9), randn(at, Hkv, ps, d, seed=seed + 19)
        args = (q, kp, vp, i32(table), i32(np.concatenate([[0], np.cumsum(nq)])), i32(nk))
        ws = torch.full((ops.varlen_workspace_size(B, T, Hq, Hkv),), 0xFF, dtype=torch.uint8, device=DEV)
        want = ops.fwd_varlen_paged(*args, workspace=ws)
        assert int(ws[:4].view(torch.int32)) > 0, "not a planned call"
        calls.append((lambda stream, args=args, ws=ws: ops.fwd_varlen_paged(*args, workspace=ws, stream=stream), want))
    torch.cuda.synchronize()
    return calls


def test_planned_calls_on_streams_of_their_own():
    calls = planned_calls()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = []
    for _ in range(20):
        for (call, want), s in zip(calls, streams):
            outs.append((call(s), want))
    torch.cuda.synchronize()
    assert ops.get_error() == ops.FA_OK
    assert all(torch.equal(o, wo) and torch.equal(l, wl) for (o, l), (wo, wl) in outs)


def test_calls_from_several_threads():
    """One thread a stream, all in the library at once (the binding lets go of the interpreter there)."""
    import threading
    calls = planned_calls()
    wrong = []

    def work(call, want):
        torch.cuda.set_device(0)
        s = torch.cuda.Stream()
        outs = [call(s) for _ in range(30)]
        s.synchronize()
        wrong.extend(1 for o, l in outs if not (torch.equal(o, want[0]) and torch.equal(l, want[1])))

    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and ops.get_error() == ops.FA_OK


def test_nothing_to_do_on_another_stream():
    side = torch.cuda.Stream()
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    o, lse = ops.fwd_varlen(q, q, q, i32([0, 0]), stream=side)
    qo, _ = ops.rope(q, None, i32([]), torch.ones(32, device=DEV), stream=side)
    assert o.shape == qo.shape == q.shape and tuple(lse.shape) == (4, 0) and ops.get_error() == ops.FA_OK
