"""Whose memory the tensors are that a call with stream= makes itself: the allocator of PyTorch hands
a block out again in the order of the stream that it was allocated on, so what a kernel on `stream`
writes must be allocated there, and what the caller gets back must know the caller's stream.

Run on the CPU: the tensors say they are on a GPU, the library and the streams are stand-ins that
record."""
import types

import pytest
import torch

from exact_io_aware_81_b200 import ops

HERE, SIDE = 1, 7   # raw handles of the current stream and of the call's
bf16, i32, f32, u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


class OnGpu(torch.Tensor):
    is_cuda = True
    device = torch.device("cuda", 0)

    def get_device(self):
        return 0

    def record_stream(self, s):
        self.users = getattr(self, "users", []) + [s.cuda_stream]


def gpu(*shape, dtype=bf16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def made(monkeypatch):
    """The tensors allocated during the test, each with the stream that was current (`.made_on`)."""
    log, now, zeros = [], [HERE], torch.zeros

    def empty(*shape, dtype=None, device=None):
        t = zeros(*shape, dtype=dtype).as_subclass(OnGpu)
        t.made_on = now[-1]
        log.append(t)
        return t

    class on_stream:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            now.append(self.s.cuda_stream)

        def __exit__(self, *a):
            now.pop()

    class Lib:
        launched = []

        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: 64

            def call(*a):
                self.launched.append((name, a[-1]))
                self.arguments = a
                return ops.FA_OK
            return call

    lib = Lib()
    lib.launched.clear()
    monkeypatch.setattr(ops, "load", lambda *a: lib)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: FakeStream(now[-1]))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, dev=None: FakeStream(h))
    monkeypatch.setattr(torch.cuda, "device", lambda d: on_stream(FakeStream(now[-1])))
    monkeypatch.setattr(ops, "_raw_stream", lambda dev: now[-1])
    monkeypatch.setattr(ops, "_current_device", lambda: 0)
    return types.SimpleNamespace(tensors=log, lib=lib)


def serving_calls():
    q, k, c, sl = gpu(8, 4, 128), gpu(8, 2, 128), gpu(3, dtype=i32), gpu(2, dtype=i32)
    pos, inv = gpu(8, dtype=i32), gpu(64, dtype=f32)
    kp, table = gpu(6, 2, 16, 128), gpu(2, 3, dtype=i32)
    state = (table, sl, gpu(6, dtype=i32))
    return {
        "fwd_varlen": lambda **kw: ops.fwd_varlen(q, k, k, c, **kw),
        "fwd_varlen_paged": lambda **kw: ops.fwd_varlen_paged(q, kp, kp, table, c, sl, **kw),
        "rope": lambda **kw: ops.rope(q, k, pos, inv, **kw),
        "rope_append": lambda **kw: ops.rope_append(q, k, k, pos, inv, kp, kp, table, c, sl, **kw),
        "pages_reserve": lambda **kw: ops.pages_reserve(*state, gpu(2, dtype=i32), 16, **kw),
        "pages_compact": lambda **kw: ops.pages_compact(*state, 16, **kw),
    }


def flat(x):
    return [t for y in x for t in flat(y)] if isinstance(x, (tuple, list)) else [x]


def check(made, call):
    got = flat(call(stream=FakeStream(SIDE)))
    assert made.tensors and made.lib.launched and all(s == SIDE for _, s in made.lib.launched)
    for t in made.tensors:
        assert t.made_on == SIDE, f"a tensor of shape {tuple(t.shape)} is the current stream's memory"
    for t in got:
        assert any(t is m for m in made.tensors) and HERE in t.users, "the caller's stream is not recorded"
    made.tensors.clear()
    made.lib.launched.clear()
    got = flat(call())
    assert all(s == HERE for _, s in made.lib.launched)
    for t in made.tensors:
        assert t.made_on == HERE and not hasattr(t, "users")


@pytest.mark.parametrize("name", ["fwd_varlen", "fwd_varlen_paged", "rope", "rope_append", "pages_reserve", "pages_compact"])
def test_what_a_serving_call_makes_is_its_streams_memory(made, name):
    check(made, serving_calls()[name])


def dense_calls():
    q, k = gpu(2, 4, 8, 128), gpu(2, 2, 8, 128)
    q8, k8, s4, s2 = gpu(2, 4, 8, 128, dtype=u8), gpu(2, 2, 8, 128, dtype=u8), gpu(4, dtype=f32), gpu(2, dtype=f32)
    qd, sl, pages, table = gpu(2, 4, 128), gpu(2, dtype=i32), gpu(6, 2, 16, 128), gpu(2, 3, dtype=i32)
    pages8 = gpu(6, 2, 16, 128, dtype=u8)
    bshd = lambda t: t.transpose(1, 2).contiguous().as_subclass(OnGpu)  # noqa: E731
    return {
        "fwd": lambda **kw: ops.fwd(q, k, k, **kw),
        "fwd_bshd": lambda **kw: ops.fwd_bshd(bshd(q), bshd(k), bshd(k), **kw),
        "fwd_window": lambda **kw: ops.fwd_window(q, k, k, 4, **kw),
        "fwd_fp8": lambda **kw: ops.fwd_fp8(q8, k8, k8, s4, s2, s2, **kw),
        "decode": lambda **kw: ops.decode(qd, k, k, sl, **kw),
        "decode_ex": lambda **kw: ops.decode_ex(qd, k, k, sl, **kw),
        "decode_paged": lambda **kw: ops.decode_paged(qd, pages, pages, table, sl, **kw),
        "decode_fp8": lambda **kw: ops.decode_fp8(qd, k8, k8, s2, s2, sl, **kw),
        "decode_paged_fp8": lambda **kw: ops.decode_paged_fp8(qd, pages8, pages8, s2, s2, table, sl, **kw),
        "merge_lse": lambda **kw: ops.merge_lse(gpu(3, 2, 4, 64, dtype=f32), gpu(3, 2, 4, dtype=f32), **kw),
        "fwd_selftest_timeout": lambda **kw: ops.fwd_selftest_timeout(q, k, k, **kw),
        "decode_selftest_timeout": lambda **kw: ops.decode_selftest_timeout(qd, k, k, sl, **kw),
    }


@pytest.mark.parametrize("name", ["fwd", "fwd_bshd", "fwd_window", "fwd_fp8", "decode", "decode_ex", "decode_paged",
                                  "decode_fp8", "decode_paged_fp8", "merge_lse", "fwd_selftest_timeout",
                                  "decode_selftest_timeout"])
def test_what_a_dense_or_decode_call_makes_is_its_streams_memory(made, name):
    check(made, dense_calls()[name])
