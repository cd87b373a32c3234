"""A reservation that the pool cannot serve, and what the step does after it: the status word that
fa_pages_reserve_ex writes keeps the appends from overwriting finished tokens."""
import pytest
import torch

from exact_io_aware_81_b200 import ops

pytestmark = pytest.mark.gpu

DEV = "cuda"
PS = 16


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


class Cache:
    """Two slots of 20 tokens that share their pages, in a pool of three pages."""

    def __init__(self, Hkv=2, d=128, fp8=False):
        g = torch.Generator().manual_seed(0)
        self.table = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
        self.lens, self.ref = i32([0, 0]), i32([0, 0, 0])
        self.status = i32([99])
        if fp8:
            self.kp, self.vp = (torch.randint(0, 127, (3, Hkv, PS, d), generator=g, dtype=torch.uint8).to(DEV) for _ in range(2))
            self.scales = dict(k_scale=torch.ones(Hkv, device=DEV), v_scale=torch.ones(Hkv, device=DEV))
        else:
            self.kp, self.vp = (torch.randn(3, Hkv, PS, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
            self.scales = {}
        ops.pages_reserve(*self.state, i32([20, 0]), PS, status=self.status)
        assert int(self.status) == ops.FA_OK
        ops.pages_fork(*self.state, i32([0]), i32([1]), PS)

    @property
    def state(self):
        return self.table, self.lens, self.ref

    def everything(self):
        return [t.clone() for t in (*self.state, self.kp, self.vp)]

    def same(self, before):
        return all(torch.equal(a, b) for a, b in zip(self.everything(), before))


def rows(T, H, d, seed=1):
    return torch.randn(T, H, d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("F", [64, 13])
@pytest.mark.parametrize("d", [64, 128])
def test_a_refused_reservation_writes_nothing(d, F, fp8):
    """Both slots grow by a token: two splits, one free page.  Without the status word the step would
    put the new rows over token 19, which the slots share."""
    if fp8 and d == 64 or F > d // 2:
        pytest.skip("E4M3 pages have d = 128, and F is at most d / 2")
    c = Cache(d=d, fp8=fp8)
    before = c.everything()
    copies = ops.pages_reserve(*c.state, i32([1, 1]), PS, status=c.status)
    ops.pages_copy(c.kp, c.vp, copies)
    q, k, v = rows(2, 4, d), rows(2, 2, d, 2), rows(2, 2, d, 3)
    q_out = torch.full_like(q, 7.0)
    cu, pos, inv = i32([0, 1, 2]), i32([20, 20]), torch.ones(F, device=DEV)
    ops.rope_append(q, k, v, pos, inv, c.kp, c.vp, c.table, cu, c.lens, q_out=q_out, status=c.status, **c.scales)
    ops.cache_append(k, v, c.kp, c.vp, c.table, cu, c.lens, status=c.status, **c.scales)
    assert int(c.status) == ops.FA_ERR_NO_PAGES
    assert ops.get_error() == ops.FA_OK, "a full pool is the caller's, not the process's"
    assert c.same(before) and (copies == -1).all() and (q_out == 7.0).all()
    # one slot gives up its place, and the step goes through
    ops.pages_free(*c.state, i32([1]), PS)
    copies = ops.pages_reserve(*c.state, i32([1, 1]), PS, status=c.status)
    ops.pages_copy(c.kp, c.vp, copies)
    got = ops.rope_append(q, k, v, pos, inv, c.kp, c.vp, c.table, cu, c.lens, q_out=q_out, status=c.status, **c.scales)
    assert int(c.status) == ops.FA_OK == ops.get_error() and c.lens.tolist() == [21, 1]
    want = ops.rope(q, None, pos, inv)[0]
    assert torch.equal(got, want)
    if not fp8:
        assert torch.equal(c.vp[int(c.table[0, 1]), :, 4], v[0]) and torch.equal(c.vp[int(c.table[1, 0]), :, 0], v[1])
    assert torch.equal(c.kp[:, :, 8:], before[3][:, :, 8:])


def test_a_length_that_cannot_be_is_refused_too():
    c = Cache()
    before = c.everything()
    copies = ops.pages_reserve(*c.state, i32([-1, 0]), PS, status=c.status)
    k = rows(1, 2, 128)
    ops.cache_append(k, k, c.kp, c.vp, c.table, i32([0, 1, 1]), c.lens, status=c.status)
    assert int(c.status) == ops.FA_ERR_DEVICE_ARG == ops.get_error() and ops.get_error() == ops.FA_OK
    assert c.same(before) and (copies == -1).all()


def test_without_a_status_word_the_error_word_has_it():
    c = Cache()
    ops.pages_reserve(*c.state, i32([1, 1]), PS)
    assert ops.get_error() == ops.FA_ERR_NO_PAGES and ops.get_error() == ops.FA_OK


def test_a_captured_step_follows_the_pool():
    """One captured step, replayed until the pool is full and once more: the last replay changes
    nothing, and after a slot was freed the same graph goes on."""
    c = Cache()
    ops.pages_free(*c.state, i32([1]), PS)
    k, q = rows(1, 2, 128), rows(1, 4, 128, 5)
    cu, pos, inv, add = i32([0, 1, 1]), i32([20]), torch.ones(64, device=DEV), i32([1, 0])
    copies = torch.empty(2, 2, dtype=torch.int32, device=DEV)
    ws = torch.empty(ops.pages_reserve_workspace_size(2, 3), dtype=torch.uint8, device=DEV)
    q_out = torch.empty_like(q)

    def step():
        ops.pages_reserve(*c.state, add, PS, copies=copies, workspace=ws, status=c.status)
        ops.pages_copy(c.kp, c.vp, copies)
        ops.rope_append(q, k, k, pos, inv, c.kp, c.vp, c.table, cu, c.lens, q_out=q_out, status=c.status)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(22, 49):
        graph.replay()
        assert int(c.status) == ops.FA_OK and c.lens.tolist() == [n, 0]
        assert torch.equal(c.vp[int(c.table[0, (n - 1) // PS]), :, (n - 1) % PS], k[0])
    before = c.everything()
    k.fill_(3.0)
    graph.replay()
    assert int(c.status) == ops.FA_ERR_NO_PAGES and c.same(before) and ops.get_error() == ops.FA_OK
    ops.pages_free(*c.state, i32([0]), PS, keep=i32([10]))
    graph.replay()
    assert int(c.status) == ops.FA_OK and c.lens.tolist() == [11, 0] and (c.vp[int(c.table[0, 0]), :, 10] == 3.0).all()


def test_status_is_checked():
    c = Cache()
    for bad in (i32([0, 0]), torch.zeros(1, device=DEV), torch.zeros(1, dtype=torch.int32), i32([[0]])):
        with pytest.raises(ValueError):
            ops.pages_reserve(*c.state, i32([1, 0]), PS, status=bad)
        with pytest.raises(ValueError):
            ops.cache_append(rows(1, 2, 128), rows(1, 2, 128), c.kp, c.vp, c.table, i32([0, 1, 1]), c.lens, status=bad)
    assert c.lens.tolist() == [20, 20]


@pytest.mark.parametrize("other", ["page", "slot", "both"])
def test_the_error_word_loses_nothing(other):
    """A full pool and a bad argument in one step: fa_get_error returns one status after another."""
    c = Cache()
    ops.pages_reserve(*c.state, i32([1, 1]), PS)                  # too few pages
    if other != "slot":
        ops.pages_copy(c.kp, c.vp, i32([[0, 7]]))                 # no such page
    if other != "page":
        ops.pages_free(*c.state, i32([9]), PS)                    # no such slot
    assert [ops.get_error() for _ in range(3)] == [ops.FA_ERR_DEVICE_ARG, ops.FA_ERR_NO_PAGES, ops.FA_OK]
    assert c.lens.tolist() == [20, 20]
