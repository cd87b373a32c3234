"""Page management (fa_pages_*) against plain lists, and against what the pages are for: every
slot's tokens, read back through its table, are the tokens it was given."""
import random

import numpy as np
import pytest
import torch

from exact_io_aware_81_b200 import ops
from oracle import serving

pytestmark = pytest.mark.gpu

DEV = "cuda"


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).to(DEV)


class Both:
    """The device state beside the plain one, with a pool whose rows hold token numbers."""

    def __init__(self, S, max_pages, num_pages, ps, d=64):
        self.ref = serving.Pages(S, max_pages, num_pages, ps)
        self.table = torch.full((S, max_pages), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(S, dtype=torch.int32, device=DEV)
        self.count = torch.zeros(num_pages, dtype=torch.int32, device=DEV)
        self.kp = torch.zeros(num_pages, 1, ps, d, dtype=torch.uint8, device=DEV)
        self.vp = torch.zeros_like(self.kp)
        self.tokens = [[] for _ in range(S)]
        self.ps, self.S = ps, S
        self.next = 0

    @property
    def state(self):
        return self.table, self.lens, self.count

    def check(self, status=ops.FA_OK):
        assert ops.get_error() == status
        assert torch.equal(self.lens.cpu(), torch.from_numpy(self.ref.lens))
        assert torch.equal(self.count.cpu(), torch.from_numpy(self.ref.ref))
        t = self.table.cpu().numpy()
        for s in range(self.S):
            h = self.ref.held(self.ref.lens[s])
            assert (t[s, :h] == self.ref.table[s, :h]).all()
            assert (t[s, h:] == -1).all()

    def contents(self):
        kp = self.kp.cpu()
        for s in range(self.S):
            n = len(self.tokens[s])
            assert n == self.ref.lens[s]
            got = serving.gather(kp, self.ref.table, s, n)[:, 0, :4].contiguous().view(torch.int32)[:, 0] if n else []
            assert list(map(int, got)) == self.tokens[s], f"slot {s}"

    def reserve(self, add):
        copies = ops.pages_reserve(*self.state, i32(add), self.ps)
        want = self.ref.reserve(add)
        if want is None:
            assert (copies == -1).all()
            return False
        assert torch.equal(copies.cpu(), torch.from_numpy(want))
        ops.pages_copy(self.kp, self.vp, copies)
        # write the new tokens where the table says
        kp = self.kp.cpu()
        for s, a in enumerate(add):
            for _ in range(a):
                p = len(self.tokens[s])
                self.tokens[s].append(self.next)
                row = torch.tensor([self.next], dtype=torch.int32).view(torch.uint8)
                kp[int(self.ref.table[s, p // self.ps]), 0, p % self.ps, :4] = row
                self.next += 1
        self.kp.copy_(kp)
        return True

    def fork(self, src, dst, lengths=None):
        ops.pages_fork(*self.state, i32(src), i32(dst), self.ps, lengths=i32(lengths) if lengths is not None else None)
        self.ref.fork(src, dst, lengths)
        for i, (s, d) in enumerate(zip(src, dst)):
            self.tokens[d] = self.tokens[s][:len(self.tokens[s]) if lengths is None else lengths[i]]

    def free(self, slots, keep=None):
        ops.pages_free(*self.state, i32(slots), self.ps, keep=i32(keep) if keep is not None else None)
        self.ref.free(slots, keep)
        for i, s in enumerate(slots):
            self.tokens[s] = self.tokens[s][:0 if keep is None else keep[i]]

    def compact(self):
        copies = ops.pages_compact(*self.state, self.ps)
        want = self.ref.compact()
        assert torch.equal(copies.cpu(), torch.from_numpy(want))
        ops.pages_copy(self.kp, self.vp, copies)
        n = int((self.count > 0).sum())
        assert (self.count[:n] > 0).all() and (self.count[n:] == 0).all()


@pytest.mark.parametrize("seed,S,mp,np_,ps", [(1, 6, 9, 40, 16), (2, 3, 5, 11, 32), (3, 40, 7, 300, 16), (4, 1, 3, 3, 48),
                                              (5, 12, 30, 250, 16)])
def test_a_random_life(seed, S, mp, np_, ps):
    r = random.Random(seed)
    b = Both(S, mp, np_, ps)
    done = {"full": 0}
    for step in range(60):
        op = r.choice(["reserve", "reserve", "fork", "free", "cut", "compact"])
        empty = [s for s in range(S) if b.ref.lens[s] == 0]
        held = [s for s in range(S) if b.ref.lens[s] > 0]
        if op == "reserve":
            add = [r.choice([0, 0, 1, 1, 5, ps, 3 * ps - 1]) for _ in range(S)]
            add = [min(a, ps * mp - int(b.ref.lens[s])) for s, a in enumerate(add)]
            if not b.reserve(add):
                done["full"] += 1
                b.check(ops.FA_ERR_NO_PAGES)
        elif op == "fork" and empty and held:
            n = r.randint(1, len(empty))
            src, dst = [r.choice(held) for _ in range(n)], r.sample(empty, n)
            b.fork(src, dst, None if r.random() < 0.5 else [r.randint(0, int(b.ref.lens[s])) for s in src])
        elif op == "free" and held:
            b.free(r.sample(held, r.randint(1, len(held))))
        elif op == "cut" and held:
            slots = r.sample(held, r.randint(1, len(held)))
            b.free(slots, [r.randint(0, int(b.ref.lens[s])) for s in slots])
        elif op == "compact":
            b.compact()
        b.check()
        b.contents()


def test_reserve_is_all_or_nothing():
    b = Both(4, 8, 10, 16)
    assert b.reserve([16 * 3, 5, 0, 16])
    b.check()
    assert not b.reserve([1, 12, 16 * 4, 16])   # 1 + 1 + 4 + 1 pages wanted, 10 - 3 - 1 - 1 free
    b.check(ops.FA_ERR_NO_PAGES)
    assert b.reserve([1, 11, 16 * 4, 0])        # 1 + 0 + 4: exactly the free ones
    b.check()
    assert not b.reserve([0, 1, 0, 0])
    b.check(ops.FA_ERR_NO_PAGES)
    assert b.reserve([0, 0, 0, 0])
    b.contents()


@pytest.mark.parametrize("add", [[-1, 0], [16 * 4 + 1, 0], [2 ** 31 - 1, 2 ** 31 - 1]])
def test_reserve_refuses_a_length(add):
    b = Both(2, 4, 20, 16)
    assert b.reserve([3, 4])
    copies = ops.pages_reserve(*b.state, i32(add), 16)
    assert (copies == -1).all()
    b.check(ops.FA_ERR_DEVICE_ARG)
    b.check()


def test_sharers_split_once_each():
    """Three slots share a partly filled page; extended together each gets its own, and the
    shared one is free afterwards.  A full shared page is never split."""
    b = Both(5, 6, 30, 16)
    b.reserve([21, 0, 0, 32, 0])
    b.fork([0, 0, 3], [1, 2, 4])
    tail = int(b.ref.table[0, 1])
    b.reserve([1, 1, 1, 1, 1])
    b.check()
    b.contents()
    assert b.ref.ref[tail] == 0
    assert b.ref.table[3, 1] == b.ref.table[4, 1] and b.ref.ref[b.ref.table[3, 1]] == 2


def test_fork_and_free_refuse():
    b = Both(6, 4, 40, 16)
    b.reserve([20, 30, 0, 0, 0, 0])
    # (source, destination, length): refused are a destination in use, a slot that does not
    # exist, a length too long or negative, a second pair for one destination, a source that is
    # also a destination; the rest happens
    for src, dst, lengths, ok in [([0, 0], [1, 2], None, [1]), ([7, 0], [3, 4], None, [1]), ([0, 0], [-1, 5], None, [1]),
                                  ([0, 1], [3, 3], [21, 5], []), ([0], [3], [-1], [])]:
        ops.pages_fork(*b.state, i32(src), i32(dst), 16, lengths=i32(lengths) if lengths else None)
        if ok:
            b.ref.fork([src[i] for i in ok], [dst[i] for i in ok])
            for i in ok:
                b.tokens[dst[i]] = list(b.tokens[src[i]])
        b.check(ops.FA_ERR_DEVICE_ARG)
    b.contents()
    b.free([2, 4, 5])
    ops.pages_fork(*b.state, i32([0, 2]), i32([2, 3]), 16)   # slot 2 as destination and source
    b.ref.fork([], [])
    # slot 2 is a destination, so the pair that reads it is refused
    b.ref.fork([0], [2])
    b.tokens[2] = list(b.tokens[0])
    b.check(ops.FA_ERR_DEVICE_ARG)
    for slots, keep, ok in [([0, 0], None, [0]), ([9, 1], [0, 7], [1]), ([1], [8], []), ([1], [-2], [])]:
        ops.pages_free(*b.state, i32(slots), 16, keep=i32(keep) if keep else None)
        if ok:
            b.ref.free([slots[i] for i in ok], [keep[i] for i in ok] if keep else None)
            for i in ok:
                b.tokens[slots[i]] = b.tokens[slots[i]][:keep[i] if keep else 0]
        b.check(ops.FA_ERR_DEVICE_ARG)
    b.contents()


@pytest.mark.parametrize("N,live", [(1, 1), (2, 1), (5, 3), (4096, 2000), (4099, 4098), (20011, 9001), (70003, 30000), (8192, 0)])
def test_compact_large_pools(N, live):
    r = np.random.RandomState(N)
    pages = r.permutation(N)[:live].astype(np.int32)
    S = 3
    cuts = np.sort(r.randint(0, live + 1, S - 1)) if live else np.zeros(S - 1, int)
    rows = np.split(pages, cuts)
    mp = max(1, max(map(len, rows)))
    p = serving.Pages(S, mp, N, 16)
    for s, row in enumerate(rows):
        p.table[s, :len(row)] = row
        p.lens[s] = 16 * len(row) - (5 if len(row) else 0)
        p.ref[row] += 1
    table, lens, count = i32(p.table), i32(p.lens), i32(p.ref)
    held = i32(p.table >= 0).bool()
    before = table.clone()
    copies = ops.pages_compact(table, lens, count, 16)
    assert ops.get_error() == ops.FA_OK
    c = copies.cpu().numpy()
    moves = int((c[:, 0] >= 0).sum())
    n = live
    assert (c[:moves, 0] >= n).all() and (c[:moves, 1] < n).all() and (c[moves:] == -1).all()
    assert (np.diff(c[:moves, 0]) > 0).all() and (np.diff(c[:moves, 1]) > 0).all()
    to = np.arange(N)
    to[c[:moves, 0]] = c[:moves, 1]
    want = before.cpu().numpy().copy()
    want[want >= 0] = to[want[want >= 0]]
    assert (table.cpu().numpy() == want).all() and held.shape == table.shape
    assert (count.cpu().numpy()[:n] == 1).all() and not count.cpu().numpy()[n:].any()


def test_many_slots_reserve():
    """More slots than one step of the sums holds, growth of nothing to many pages."""
    S, ps, mp = 2500, 16, 40
    r = np.random.RandomState(0)
    p = serving.Pages(S, mp, 40000, ps)
    table, lens, count = i32(p.table), i32(p.lens), i32(p.ref)
    for _ in range(3):
        add = r.choice([0, 1, 7, 33, 200], S, p=[0.3, 0.3, 0.2, 0.15, 0.05])
        add = np.minimum(add, ps * mp - p.lens)
        copies = ops.pages_reserve(table, lens, count, i32(add), ps)
        assert torch.equal(copies.cpu(), torch.from_numpy(p.reserve(add)))
        assert ops.get_error() == ops.FA_OK
        assert (table.cpu().numpy() == p.table).all() and (lens.cpu().numpy() == p.lens).all()
        assert (count.cpu().numpy() == p.ref).all()


def test_own_workspace_on_another_stream():
    """reserve and compact with workspaces of their own on a busy stream, while the current
    stream allocates and writes as much."""
    S, ps, mp, N = 300, 16, 20, 4000
    r = np.random.RandomState(1)
    p = serving.Pages(S, mp, N, ps)
    table, lens, count = i32(p.table), i32(p.lens), i32(p.ref)
    add, gone = r.randint(0, 150, S), np.arange(0, S, 3)
    side = torch.cuda.Stream()
    add_d, gone_d = i32(add), i32(gone)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms
    c1 = ops.pages_reserve(table, lens, count, add_d, ps, stream=side)
    ops.pages_free(table, lens, count, gone_d, ps, stream=side)
    c2 = ops.pages_compact(table, lens, count, ps, stream=side)
    sizes = [ops.pages_reserve_workspace_size(S, N), ops.pages_compact_workspace_size(N)]
    fill = [torch.full((n,), 0x11, dtype=torch.uint8, device=DEV) for n in sizes * 4]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert ops.get_error() == ops.FA_OK and len(fill) == 8
    assert torch.equal(c1.cpu(), torch.from_numpy(p.reserve(add)))
    p.free(gone)
    assert torch.equal(c2.cpu(), torch.from_numpy(p.compact()))
    assert (lens.cpu().numpy() == p.lens).all() and (count.cpu().numpy() == p.ref).all()
    for s in range(S):
        h = p.held(p.lens[s])
        assert (table.cpu().numpy()[s, :h] == p.table[s, :h]).all()


@pytest.mark.parametrize("shape,dtype", [((9, 1, 16, 64), torch.uint8), ((7, 3, 48, 64), torch.bfloat16),
                                         ((12, 8, 64, 128), torch.bfloat16), ((600, 2, 16, 128), torch.uint8)])
def test_copy(shape, dtype):
    g = torch.Generator(DEV).manual_seed(1)
    kp, vp = (torch.randint(0, 120, shape, generator=g, device=DEV).to(dtype) for _ in range(2))
    N = shape[0]
    n = N // 3
    perm = torch.randperm(N, generator=torch.Generator().manual_seed(2))
    pairs = torch.stack([perm[:n], perm[n:2 * n]], 1).to(torch.int32)
    rows = torch.full((2 * n + 1, 2), -1, dtype=torch.int32)
    rows[1::2] = pairs
    wk, wv = kp.clone(), vp.clone()
    wk[pairs[:, 1].long()] = kp[pairs[:, 0].long()]
    wv[pairs[:, 1].long()] = vp[pairs[:, 0].long()]
    k1 = kp.clone()
    ops.pages_copy(k1, None, rows.to(DEV))
    assert torch.equal(k1, wk)
    ops.pages_copy(kp, vp, rows.to(DEV))
    assert torch.equal(kp, wk) and torch.equal(vp, wv) and ops.get_error() == ops.FA_OK


def test_copy_reports_a_page_outside_the_pool():
    kp = torch.arange(4 * 16 * 64, device=DEV).to(torch.uint8).view(4, 1, 16, 64).contiguous()
    want = kp.clone()
    want[1] = kp[0]
    ops.pages_copy(kp, None, i32([[4, 2], [0, 1], [3, -1], [2, 9]]))
    assert ops.get_error() == ops.FA_ERR_DEVICE_ARG
    assert torch.equal(kp, want)


def test_captured_and_replayed():
    """A captured step (free, fork, reserve, copy) replayed gives what the calls give, and does
    not depend on what else ran since."""
    b = Both(8, 6, 40, 16)
    b.reserve([21, 50, 0, 0, 0, 0, 0, 0])
    src, dst, add = i32([0, 0, 1]), i32([2, 3, 4]), i32([0, 0, 1, 17, 2, 0, 0, 0])
    copies = torch.empty(8, 2, dtype=torch.int32, device=DEV)
    ws = torch.empty(ops.pages_reserve_workspace_size(8, 40), dtype=torch.uint8, device=DEV)

    def step():
        ops.pages_free(*b.state, dst, 16)
        ops.pages_fork(*b.state, src, dst, 16)
        ops.pages_reserve(*b.state, add, 16, copies=copies, workspace=ws)
        ops.pages_copy(b.kp, b.vp, copies)

    step()
    want = [t.clone() for t in (*b.state, copies, b.kp)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ws.fill_(0x5A)
    for _ in range(3):
        graph.replay()
    assert ops.get_error() == ops.FA_OK
    for t, w in zip((*b.state, copies, b.kp), want):
        assert torch.equal(t, w)
