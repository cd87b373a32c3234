"""Host side of the operators around the paged attention: refusals that need no GPU, and the
plain restatements the GPU tests compare with, fixed by something other than themselves."""
import math

import numpy as np
import pytest
import torch

from exact_io_aware_81_b200 import build, ops
from oracle import serving

FAKE = 0x10000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return ops.load()


def _rope(lib, **kw):
    a = dict(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, pos=FAKE, inv=FAKE, axes=None, T=4, Hq=4, Hkv=2, d=128, F=64, A=1,
             qs=512, ks=256, qos=512, kos=256, dt=ops.FA_BF16)
    a.update(kw)
    return lib.fa_rope(a["q"], a["k"], a["qo"], a["ko"], a["pos"], a["inv"], a["axes"], a["T"], a["Hq"], a["Hkv"],
                       a["d"], a["F"], a["A"], a["qs"], a["ks"], a["qos"], a["kos"], a["dt"], 0, 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), ops.FA_ERR_INVALID), (dict(ko=None), ops.FA_ERR_INVALID), (dict(pos=None), ops.FA_ERR_INVALID),
    (dict(inv=None), ops.FA_ERR_INVALID), (dict(T=0), ops.FA_ERR_INVALID), (dict(Hq=0, Hkv=0), ops.FA_ERR_INVALID),
    (dict(Hq=-1), ops.FA_ERR_INVALID), (dict(F=0), ops.FA_ERR_INVALID), (dict(F=65), ops.FA_ERR_INVALID),
    (dict(A=0), ops.FA_ERR_INVALID), (dict(dt=2), ops.FA_ERR_INVALID), (dict(d=96, F=8), ops.FA_ERR_UNSUPPORTED),
    (dict(qs=511), ops.FA_ERR_UNSUPPORTED), (dict(qs=516), ops.FA_ERR_UNSUPPORTED), (dict(kos=128), ops.FA_ERR_UNSUPPORTED),
    (dict(k=FAKE + 8), ops.FA_ERR_UNSUPPORTED),
])
def test_rope_rejects(lib, kw, status):
    assert _rope(lib, **kw) == status
    assert lib.fa_last_error_message().decode() != ""


def _append(lib, **kw):
    a = dict(k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, ks=None, vs=None, bt=FAKE, cu=FAKE, sl=FAKE, T=4, B=2, Hkv=2, np=10,
             ps=64, mp=5, d=128, kst=256, vst=256)
    a.update(kw)
    return lib.fa_cache_append(a["k"], a["v"], a["kp"], a["vp"], a["ks"], a["vs"], a["bt"], a["cu"], a["sl"], a["T"],
                               a["B"], a["Hkv"], a["np"], a["ps"], a["mp"], a["d"], a["kst"], a["vst"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), ops.FA_ERR_INVALID), (dict(v=None), ops.FA_ERR_INVALID), (dict(vp=None), ops.FA_ERR_INVALID),
    (dict(bt=None), ops.FA_ERR_INVALID), (dict(cu=None), ops.FA_ERR_INVALID), (dict(sl=None), ops.FA_ERR_INVALID),
    (dict(ks=FAKE), ops.FA_ERR_INVALID), (dict(T=0), ops.FA_ERR_INVALID), (dict(B=0), ops.FA_ERR_INVALID),
    (dict(Hkv=0), ops.FA_ERR_INVALID), (dict(np=0), ops.FA_ERR_INVALID), (dict(mp=-1), ops.FA_ERR_INVALID),
    (dict(ps=24), ops.FA_ERR_UNSUPPORTED), (dict(d=32), ops.FA_ERR_UNSUPPORTED),
    (dict(ks=FAKE, vs=FAKE, d=64), ops.FA_ERR_UNSUPPORTED), (dict(vst=257), ops.FA_ERR_UNSUPPORTED),
    (dict(kp=FAKE + 4), ops.FA_ERR_UNSUPPORTED),
])
def test_cache_append_rejects(lib, kw, status):
    assert _append(lib, **kw) == status


def test_rope_append_rejects(lib):
    def call(q=FAKE, qo=FAKE, inv=FAKE, v=FAKE, F=64, T=4):
        return lib.fa_rope_append(q, FAKE, v, qo, FAKE, inv, None, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, T, 2, 4, 2,
                                  10, 64, 5, 128, F, 1, 512, 256, 256, 512, 0, None)
    for kw in (dict(q=None), dict(qo=None), dict(inv=None), dict(v=None), dict(F=0), dict(T=-1)):
        assert call(**kw) == ops.FA_ERR_INVALID


STATE = dict(bt=FAKE, sl=FAKE, rc=FAKE, S=4, mp=8, np=32, ps=16)


@pytest.mark.parametrize("kw,status", [
    (dict(bt=None), ops.FA_ERR_INVALID), (dict(sl=None), ops.FA_ERR_INVALID), (dict(rc=None), ops.FA_ERR_INVALID),
    (dict(S=0), ops.FA_ERR_INVALID), (dict(mp=0), ops.FA_ERR_INVALID), (dict(np=-3), ops.FA_ERR_INVALID),
    (dict(ps=0), ops.FA_ERR_INVALID), (dict(ps=20), ops.FA_ERR_UNSUPPORTED), (dict(mp=1 << 28), ops.FA_ERR_UNSUPPORTED),
    (dict(np=1 << 21), ops.FA_ERR_UNSUPPORTED), (dict(S=(1 << 20) + 1), ops.FA_ERR_UNSUPPORTED),
])
def test_page_calls_reject_a_state(lib, kw, status):
    a = dict(STATE, **kw)
    s, z = (a["bt"], a["sl"], a["rc"]), (a["S"], a["mp"], a["np"], a["ps"])
    big = 1 << 40
    assert lib.fa_pages_fork(*s, FAKE, FAKE, None, 2, *z, None) == status
    assert lib.fa_pages_free(*s, FAKE, None, 2, *z, None) == status
    assert lib.fa_pages_reserve(*s, FAKE, FAKE, *z, FAKE, big, None) == status
    assert lib.fa_pages_compact(*s, FAKE, *z, FAKE, big, None) == status


def test_page_calls_reject_the_rest(lib):
    s, z = (FAKE, FAKE, FAKE), (4, 8, 32, 16)
    bad = ops.FA_ERR_INVALID
    assert lib.fa_pages_fork(*s, None, FAKE, None, 2, *z, None) == bad
    assert lib.fa_pages_fork(*s, FAKE, FAKE, None, 0, *z, None) == bad
    assert lib.fa_pages_fork(*s, FAKE, FAKE, None, 70000, *z, None) == ops.FA_ERR_UNSUPPORTED
    assert lib.fa_pages_free(*s, None, None, 2, *z, None) == bad
    assert lib.fa_pages_free(*s, FAKE, None, -1, *z, None) == bad
    assert lib.fa_pages_reserve(*s, None, FAKE, *z, FAKE, 1 << 40, None) == bad
    assert lib.fa_pages_reserve(*s, FAKE, None, *z, FAKE, 1 << 40, None) == bad
    assert lib.fa_pages_compact(*s, None, *z, FAKE, 1 << 40, None) == bad
    assert lib.fa_pages_copy(None, FAKE, FAKE, 1, 4, 4096, None) == bad
    assert lib.fa_pages_copy(FAKE, FAKE, None, 1, 4, 4096, None) == bad
    assert lib.fa_pages_copy(FAKE, FAKE, FAKE, -1, 4, 4096, None) == bad
    assert lib.fa_pages_copy(FAKE, FAKE, FAKE, 1, 4, 4100, None) == ops.FA_ERR_UNSUPPORTED
    assert lib.fa_pages_copy(FAKE + 8, FAKE, FAKE, 1, 4, 4096, None) == ops.FA_ERR_UNSUPPORTED
    assert lib.fa_pages_copy(FAKE, FAKE, FAKE, 1, 1 << 20, 1 << 30, None) == ops.FA_ERR_UNSUPPORTED
    assert lib.fa_pages_copy(FAKE, FAKE, FAKE, 1, 1, 1 << 45, None) == ops.FA_ERR_UNSUPPORTED


def test_page_workspaces_without_a_gpu(lib):
    assert lib.fa_pages_reserve_workspace_size(4, 32) == 512
    assert lib.fa_pages_reserve_workspace_size(0, 32) == 0
    assert lib.fa_pages_compact_workspace_size(100) == 256 + 2 * 512
    assert lib.fa_pages_compact_workspace_size(0) == 0


def test_binding_refuses_cpu_tensors(lib):
    z = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.rope(z, z, i, torch.ones(32))
    with pytest.raises(ValueError):
        ops.rope(None, None, i, torch.ones(32))
    with pytest.raises(TypeError):
        ops.rope([1], None, i, torch.ones(32))
    with pytest.raises(ValueError):
        ops.cache_append(z, z, z[None], z[None], i[None], i, i)
    with pytest.raises(ValueError):
        ops.pages_reserve(i[None], i[:1], i, i[:1], 16)
    with pytest.raises(ValueError):
        ops.pages_copy(z[None], None, i[None])


# ------------------------------------------------------------- the plain restatements

@pytest.mark.parametrize("interleaved", [False, True])
def test_plain_rope_is_a_complex_product(interleaved):
    """Each pair as a complex number times e^{ia}; inverse undoes it; norms are kept."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 3, 16, generator=g, dtype=torch.float64)
    pos = torch.randint(0, 1000, (2, 5), generator=g, dtype=torch.int32)
    inv = torch.rand(6, generator=g)
    axes = torch.tensor([0, 1, 1, 0, 1, 0], dtype=torch.int32)
    y = serving.rope(x, pos, inv, axes, interleaved)
    a = pos.double()[axes.long()].T * inv.double()
    z = torch.polar(torch.ones_like(a), a)[:, None]
    i, j = (slice(0, 12, 2), slice(1, 12, 2)) if interleaved else (slice(0, 6), slice(6, 12))
    w = torch.complex(x[..., i], x[..., j]) * z
    assert torch.allclose(torch.complex(y[..., i], y[..., j]), w, atol=1e-12)
    assert torch.equal(y[..., 12:], x[..., 12:])
    assert torch.allclose(serving.rope(y, pos, inv, axes, interleaved, inverse=True), x, atol=1e-12)


def test_rotated_scores_depend_on_distance_only():
    x, y = torch.randn(2, 1, 1, 16, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    inv = torch.rand(8)
    at = lambda t, p: serving.rope(t, torch.tensor([p], dtype=torch.int32), inv)  # noqa: E731
    a = (at(x, 105) * at(y, 100)).sum()
    assert torch.allclose(a, (at(x, 5) * at(y, 0)).sum(), atol=1e-10)


def test_plain_attention_is_the_library_routine():
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(n, h, 16, generator=g, dtype=torch.float64) for n, h in ((5, 4), (9, 2), (9, 2)))
    o, lse = serving.attention(q, k, v, 0.3, True, window=4)
    last = torch.arange(5)[:, None] + 4
    j = torch.arange(9)[None]
    mask = (j <= last) & (j > last - 4)
    ref = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.transpose(0, 1).repeat_interleave(2, 0), v.transpose(0, 1).repeat_interleave(2, 0),
        attn_mask=mask, scale=0.3)
    assert torch.allclose(o, ref.transpose(0, 1), atol=1e-12)
    o, lse = serving.attention(q, k[:2], v[:2], 0.3, True)   # rows 0-2 see nothing
    assert (o[:3] == 0).all() and (lse[:, :3] == -math.inf).all() and torch.isfinite(lse[:, 3:]).all()
    assert torch.allclose(o[3, 0], v[0, 0])


def test_plain_pages_by_hand():
    p = serving.Pages(3, 4, 6, 16)
    assert (p.reserve([20, 0, 5]) == -1).all()
    assert p.table.tolist() == [[0, 1, -1, -1], [-1] * 4, [2, -1, -1, -1]] and p.ref.tolist() == [1, 1, 1, 0, 0, 0]
    p.fork([0], [1], [18])
    assert p.table[1].tolist() == [0, 1, -1, -1] and p.ref.tolist() == [2, 2, 1, 0, 0, 0] and p.lens.tolist() == [20, 18, 5]
    assert p.reserve([0, 1, 0]).tolist() == [[-1, -1], [1, 3], [-1, -1]]
    assert p.table[1].tolist() == [0, 3, -1, -1] and p.ref.tolist() == [2, 1, 1, 1, 0, 0]
    assert p.reserve([64, 0, 0]) is None
    p.free([0], [3])
    assert p.ref.tolist() == [2, 0, 1, 1, 0, 0]
    assert p.compact().tolist() == [[3, 1], [-1, -1], [-1, -1]]
    assert p.table[1].tolist() == [0, 1, -1, -1] and p.ref.tolist() == [2, 1, 1, 0, 0, 0]


def test_plain_token_rows():
    rows = serving.token_rows(np.array([[4, 2], [7, 9]]), [0, 2, 3], [17, 1], 16, 4)
    assert rows == [(4, 15), (2, 0), (7, 0), None]
