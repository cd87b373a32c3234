"""Python integers that no C int holds, on their way into the library (on the CPU: the library is a
stand-in that records what it is given, as ctypes would pass it)."""
import ctypes
import sys

import pytest

from exact_io_aware_81_b200 import ops
from test_binding_streams import dense_calls, gpu, i32, made, serving_calls  # noqa: F401


def passed(made, at):
    """The integer at place `at` from the end, after the conversion of the library's signature."""
    name, kind = made.lib.launched[-1][0], None
    kind = ops.SIGNATURES[name][1][at]
    assert kind is ctypes.c_int
    return kind(made.lib.arguments[at]).value


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 40 + 1, sys.maxsize])
@pytest.mark.parametrize("name,at", [("fwd", -3), ("fwd_bshd", -3), ("fwd_fp8", -3), ("fwd_varlen", -5),
                                     ("fwd_varlen_paged", -5)])
def test_a_window_longer_than_an_int_is_a_long_window(made, name, at, window):  # noqa: F811
    call = {**dense_calls(), **serving_calls()}[name]
    call(causal=True, window=window)
    assert passed(made, at) == 2 ** 31 - 1


@pytest.mark.parametrize("name", ["fwd_varlen", "fwd_varlen_paged"])
@pytest.mark.parametrize("window", [-1, -2 ** 31, -2 ** 32 + 5])
def test_a_negative_window_stays_negative(made, name, window):  # noqa: F811
    serving_calls()[name](causal=True, window=window)
    assert passed(made, -5) < 0


@pytest.mark.parametrize("size,as_int", [(16, 16), (2 ** 32 + 16, 2 ** 31 - 1), (-2 ** 32 + 16, -2 ** 31)])
def test_a_page_size_is_not_cut(made, size, as_int):  # noqa: F811
    state = gpu(2, 3, dtype=i32), gpu(2, dtype=i32), gpu(6, dtype=i32)
    one = gpu(1, dtype=i32)
    for call, at in ((lambda: ops.pages_reserve(*state, gpu(2, dtype=i32), size), -4),
                     (lambda: ops.pages_compact(*state, size), -4),
                     (lambda: ops.pages_fork(*state, one, one, size), -2), (lambda: ops.pages_free(*state, one, size), -2)):
        call()
        assert passed(made, at) == as_int
