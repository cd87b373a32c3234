"""Rotary positions (fa_rope), filling a paged cache (fa_cache_append) and both in one launch
(fa_rope_append) against a 64-bit restatement.

Tolerances.  The angle enters sincospif as a 32-bit number of half turns of at most 1, so it
is off by at most 2^-25 half turns = pi 2^-25 < 2^-23 rad; sincospif's own error and the three
32-bit operations of x c - y s add at most 2^-22 (|x| + |y|) more: delta = 2^-21 (|x| + |y|)
bounds the error before the one rounding to the output's type, which adds half a step,
finfo.eps / 2 relative.
"""
import pytest
import torch

from exact_io_aware_81_b200 import ops
from oracle import serving

pytestmark = pytest.mark.gpu

DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def tables(F, A, seed):
    g = torch.Generator().manual_seed(seed)
    inv = (10000.0 ** (-torch.arange(F, dtype=torch.float64) / F)).float()
    axes = torch.randint(0, A, (F,), generator=g, dtype=torch.int32)
    return inv, axes


def delta(x, F, interleaved):
    """2^-21 (|x| + |y|) for both elements of each pair, 0 for copied elements."""
    a = x.double().abs()
    out = torch.zeros_like(a)
    if interleaved:
        s = a[..., 0:2 * F:2] + a[..., 1:2 * F:2]
        out[..., 0:2 * F:2] = s
        out[..., 1:2 * F:2] = s
    else:
        s = a[..., :F] + a[..., F:2 * F]
        out[..., :F] = s
        out[..., F:2 * F] = s
    return out * 2.0 ** -21


def check(got, ref, x, F, interleaved, dtype):
    d = delta(x.cpu(), F, interleaved)
    err = (got.cpu().double() - ref).abs()
    tol = HALF[dtype] * (ref.abs() + d) + d
    assert (err <= tol).all(), ((err - tol).max().item(), err.max().item())
    assert torch.equal(got[..., 2 * F:].cpu(), x[..., 2 * F:].cpu().to(dtype)), "copied elements changed"


CASES = [  # (T, Hq, Hkv, d, F, A, interleaved, dtype)
    (1, 32, 8, 128, 64, 1, False, torch.bfloat16),
    (7, 32, 8, 128, 64, 3, False, torch.bfloat16),
    (300, 6, 2, 128, 64, 3, True, torch.bfloat16),
    (129, 3, 1, 64, 32, 2, False, torch.bfloat16),
    (65, 5, 5, 64, 32, 4, True, torch.float32),
    (33, 8, 2, 128, 32, 2, False, torch.float32),   # partial rotary
    (33, 8, 2, 128, 32, 1, True, torch.bfloat16),
    (50, 4, 4, 128, 12, 3, False, torch.bfloat16),  # frequencies that fill no whole chunk
    (50, 4, 4, 128, 13, 3, True, torch.bfloat16),
    (41, 4, 2, 64, 1, 1, False, torch.float32),
    (41, 4, 2, 64, 31, 2, True, torch.float32),
    (3000, 2, 1, 64, 32, 1, False, torch.bfloat16),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,d,F,A,inter,dtype", CASES)
def test_rope_matches(T, Hq, Hkv, d, F, A, inter, dtype, inverse):
    g = torch.Generator().manual_seed(T + d + F)
    q, k = torch.randn(T, Hq, d, generator=g).to(dtype), torch.randn(T, Hkv, d, generator=g).to(dtype)
    pos = torch.randint(-50, 1 << 22, (A, T), generator=g, dtype=torch.int32)
    pos[:, 0] = 0
    inv, axes = tables(F, A, 5)
    qo, ko = ops.rope(q.to(DEV), k.to(DEV), pos.to(DEV), inv.to(DEV), axes.to(DEV), interleaved=inter, inverse=inverse)
    assert ops.get_error() == ops.FA_OK
    for got, x in ((qo, q), (ko, k)):
        check(got, serving.rope(x, pos, inv, axes, inter, inverse), x, F, inter, dtype)


def test_rope_far_positions():
    """The largest positions, at a frequency of one radian per position."""
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 16777217], dtype=torch.int32)
    x = torch.randn(4, 2, 128, generator=torch.Generator().manual_seed(1))
    inv = torch.linspace(1.0, 0.25, 64)
    qo, _ = ops.rope(x.to(DEV), None, pos.to(DEV), inv.to(DEV))
    assert ops.get_error() == ops.FA_OK
    check(qo, serving.rope(x, pos, inv), x, 64, False, torch.float32)


@pytest.mark.parametrize("inter,F", [(False, 64), (True, 64), (False, 24), (True, 21)])
def test_rope_in_place_strided_and_one_sided(inter, F):
    """q and k as slices of one fused projection, rotated in place; only k; only q."""
    T, Hq, Hkv, d = 77, 4, 2, 128
    qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32) * 37
    inv, _ = tables(F, 1, 5)
    buf = qkv.to(DEV)
    q, k = buf[:, :Hq], buf[:, Hq:Hq + Hkv]
    qo, ko = ops.rope(q, k, pos.to(DEV), inv.to(DEV), interleaved=inter, q_out=q, k_out=k)
    assert qo is q and ko is k and ops.get_error() == ops.FA_OK
    assert torch.equal(buf[:, Hq + Hkv:].cpu(), qkv[:, Hq + Hkv:]), "the values were touched"
    check(q, serving.rope(qkv[:, :Hq], pos, inv, None, inter), qkv[:, :Hq], F, inter, torch.bfloat16)
    check(k, serving.rope(qkv[:, Hq:Hq + Hkv], pos, inv, None, inter), qkv[:, Hq:Hq + Hkv], F, inter, torch.bfloat16)
    src = qkv.to(DEV)
    none, only_k = ops.rope(None, src[:, Hq:Hq + Hkv], pos.to(DEV), inv.to(DEV), interleaved=inter)
    assert none is None and torch.equal(only_k, k)
    only_q, none = ops.rope(src[:, :Hq], None, pos.to(DEV), inv.to(DEV), interleaved=inter)
    assert none is None and torch.equal(only_q, q)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_inverse_is_the_gradient(inter):
    """<g, R x> has the gradient R^T g in x: against the formula (a 64-bit autograd of the
    rotation) and against differences of the kernel's own fp32 output.  Differences: the map is
    linear, so (f(x + h e) - f(x - h e)) / 2h is exact but for the fp32 errors of f; f sums
    2 pairs' values of magnitude < 8 with relative error < 2^-21 each, so with h = 1 the
    quotient is off by less than 64 * 2^-21 < 1e-4."""
    T, H, d, F = 5, 2, 64, 32
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, H, d, generator=g)
    w = torch.randn(T, H, d, generator=g)
    pos = torch.randint(0, 100000, (T,), generator=g, dtype=torch.int32)
    inv, _ = tables(F, 1, 5)
    back, _ = ops.rope(w.to(DEV), None, pos.to(DEV), inv.to(DEV), interleaved=inter, inverse=True)
    xd = x.double().requires_grad_()
    ang = pos.double()[:, None] * inv.double()
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    a, b = (xd[..., 0::2], xd[..., 1::2]) if inter else (xd[..., :F], xd[..., F:])
    y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2) if inter else torch.cat([a * c - b * s, a * s + b * c], -1)
    (y * w.double()).sum().backward()
    check(back, xd.grad, w, F, inter, torch.float32)
    for t, h, i in ((0, 0, 0), (2, 1, 33), (4, 0, 63)):
        e = torch.zeros_like(x)
        e[t, h, i] = 1.0
        f = [(ops.rope(z.to(DEV), None, pos.to(DEV), inv.to(DEV), interleaved=inter)[0].cpu().double() * w.double())
             for z in (x + e, x - e)]
        assert abs((f[0] - f[1]).sum().item() / 2 - back[t, h, i].item()) < 1e-4


def test_rope_reports_a_bad_axis():
    q = torch.randn(3, 2, 64, device=DEV, dtype=torch.bfloat16)
    inv, _ = tables(32, 1, 5)
    axes = torch.zeros(32, dtype=torch.int32)
    pos = torch.arange(6, dtype=torch.int32).reshape(2, 3)
    good, _ = ops.rope(q, None, pos.to(DEV), inv.to(DEV), axes.to(DEV))
    axes[7] = 2
    axes[9] = -1
    got, _ = ops.rope(q, None, pos.to(DEV), inv.to(DEV), axes.to(DEV))
    assert ops.get_error() == ops.FA_ERR_DEVICE_ARG and ops.get_error() == ops.FA_OK
    assert torch.equal(got, good)  # read as axis 0


# ------------------------------------------------------------------- filling the pages

def make_append(lens_new, contexts, Hkv, d, ps, seed, fp8, spare=3, pad=0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens_new)
    T = sum(lens_new) + pad
    cu = torch.tensor([0] + lens_new).cumsum(0).to(torch.int32)
    sl = torch.tensor([n + c for n, c in zip(lens_new, contexts)], dtype=torch.int32)
    need = [-(-int(x) // ps) for x in sl]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g)
    table = torch.full((B, max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    k, v = (torch.randn(T, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
    if fp8:
        pools = [torch.randint(0, 127, (total, Hkv, ps, d), generator=g, dtype=torch.uint8) for _ in range(2)]
        scales = [torch.rand(Hkv, generator=g) * 0.01 + 0.002 for _ in range(2)]
    else:
        pools = [torch.randn(total, Hkv, ps, d, generator=g).to(torch.bfloat16) for _ in range(2)]
        scales = [None, None]
    return k, v, pools, scales, table, cu, sl, T


APPENDS = [  # (new tokens, cached tokens, Hkv, d, page size)
    ([1] * 5, [0, 15, 16, 100, 31], 8, 128, 16),
    ([1], [0], 1, 64, 16),
    ([0, 3, 0, 0, 70, 1, 0], [5, 0, 0, 64, 63, 0, 0], 2, 128, 64),
    ([130, 1, 47], [0, 47, 1], 4, 64, 48),
    ([1] * 70 + [9] * 30, list(range(100)), 1, 64, 32),
    ([2] * 1100, [0] * 1100, 1, 64, 16),   # more sequences than one search step covers
]


def device(*ts):
    return [t.to(DEV) if t is not None else None for t in ts]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("new,ctx,Hkv,d,ps", APPENDS, ids=[f"b{len(c[0])}d{c[3]}p{c[4]}" for c in APPENDS])
def test_cache_append(new, ctx, Hkv, d, ps, fp8):
    d = 128 if fp8 else d
    k, v, pools, scales, table, cu, sl, T = make_append(new, ctx, Hkv, d, ps, len(new), fp8, pad=3)
    kp, vp = device(*pools)
    ops.cache_append(*device(k, v), kp, vp, *device(table, cu, sl), *device(*scales))
    assert ops.get_error() == ops.FA_OK
    rows = serving.token_rows(table, cu, sl, ps, T)
    for got, pool, x, sc in ((kp, pools[0], k, scales[0]), (vp, pools[1], v, scales[1])):
        want = pool.clone()
        src = serving.e4m3_bytes(x.float() * (1 / sc)[:, None]) if fp8 else x
        for t, at in enumerate(rows):
            if at is not None:
                want[at[0], :, at[1]] = src[t]
        assert torch.equal(got.cpu(), want)  # every other row as it was


def test_cache_append_fp8_saturates_and_keeps_nan():
    k = torch.zeros(1, 1, 128)
    k[0, 0, :8] = torch.tensor([1e30, -1e30, float("inf"), -float("inf"), float("nan"), 500.0, -449.0, 2.0 ** -11])
    k = k.to(torch.bfloat16)
    pool = torch.zeros(1, 1, 16, 128, dtype=torch.uint8)
    kp, vp = device(pool, pool.clone())
    one = torch.ones(1)
    ops.cache_append(*device(k, k), kp, vp, *device(torch.zeros(1, 1, dtype=torch.int32),
                     torch.tensor([0, 1], dtype=torch.int32), torch.tensor([1], dtype=torch.int32), one, one))
    b = kp.cpu()[0, 0, 0, :8].tolist()
    assert b[:4] == [0x7E, 0xFE, 0x7E, 0xFE] and b[4] & 0x7F == 0x7F and b[5:] == [0x7E, 0xFE, 0x00]


@pytest.mark.parametrize("fp8,F,inter", [(False, 64, False), (False, 64, True), (False, 20, False), (True, 64, False),
                                         (True, 64, True), (True, 13, True)])
@pytest.mark.parametrize("new,ctx", [([1] * 4, [0, 3, 16, 200]), ([40, 0, 129], [7, 20, 0])])
def test_rope_append(new, ctx, fp8, F, inter):
    Hq, Hkv, d, ps, A = 8, 2, 128, 32, 2
    k, v, pools, scales, table, cu, sl, T = make_append(new, ctx, Hkv, d, ps, 9, fp8, pad=2)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(T, Hq, d, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 100000, (A, T), generator=g, dtype=torch.int32)
    inv, axes = tables(F, A, 6)
    kp, vp = device(*pools)
    qo = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    ops.rope_append(*device(q, k, v, pos, inv), kp, vp, *device(table, cu, sl, axes), interleaved=inter,
                    k_scale=scales[0].to(DEV) if fp8 else None, v_scale=scales[1].to(DEV) if fp8 else None, q_out=qo)
    assert ops.get_error() == ops.FA_OK
    n = int(cu[-1])
    check(qo[:n], serving.rope(q[:n], pos[:, :n], inv, axes, inter), q[:n], F, inter, torch.bfloat16)
    assert (qo[n:] == 7.0).all(), "padding rows were written"
    # what the pages hold: rotated keys within half a step, values exactly, the rest untouched
    rows = serving.token_rows(table, cu, sl, ps, T)
    rk = serving.rope(k[:n], pos[:, :n], inv, axes, inter)
    dk = delta(k[:n], F, inter)
    kc, vc = kp.cpu(), vp.cpu()
    want_v, touched = pools[1].clone(), torch.zeros(pools[0].shape[:3], dtype=torch.bool)
    for t in range(n):
        pg, r = rows[t]
        want_v[pg, :, r] = serving.e4m3_bytes(v[t].float() * (1 / scales[1])[:, None]) if fp8 else v[t]
        touched[pg, :, r] = True
        if fp8:
            got = kc[pg, :, r].view(torch.float8_e4m3fn).double()
            ref, dd = rk[t] / scales[0].double()[:, None], dk[t] / scales[0].double()[:, None]
            ref = ref.clamp(-448, 448)
            # half a step of E4M3 (2^-4 relative, 2^-10 among subnormals), the scaling's two roundings
            tol = 2.0 ** -4 * (ref.abs() + dd) + 2.0 ** -10 + dd + 2.0 ** -23 * ref.abs()
            assert ((got - ref).abs() <= tol).all()
        else:
            got = kc[pg, :, r].double()
            assert ((got - rk[t]).abs() <= 2.0 ** -8 * (rk[t].abs() + dk[t]) + dk[t]).all()
    assert torch.equal(vc, want_v)
    assert torch.equal(kc[~touched], pools[0][~touched])
    if not fp8:  # the same bits as the two calls it replaces
        ko = ops.rope(None, k.to(DEV), pos.to(DEV), inv.to(DEV), axes.to(DEV), interleaved=inter)[1]
        k2, v2 = device(*pools)
        ops.cache_append(ko, v.to(DEV), k2, v2, *device(table, cu, sl))
        assert torch.equal(k2, kp) and torch.equal(v2, vp)


def test_append_reports_what_it_cannot_place():
    """A page outside the pool, a length that does not hold the new tokens, a position behind
    the table: those tokens are not written, the others are."""
    k, v, pools, _, table, cu, sl, T = make_append([2, 2, 2, 2], [0, 14, 0, 30], 1, 64, 16, 1, False)
    bad_table, bad_sl = table.clone(), sl.clone()
    bad_table[0, 0] = pools[0].shape[0]   # outside the pool
    bad_sl[1] = 1                         # two new tokens in a length of one
    bad_sl[3] = 16 * table.shape[1] + 1   # the last token lies behind the table
    kp, vp = device(*pools)
    ops.cache_append(*device(k, v), kp, vp, *device(bad_table, cu, bad_sl))
    assert ops.get_error() == ops.FA_ERR_DEVICE_ARG and ops.get_error() == ops.FA_OK
    want = pools[0].clone()
    want[table[2, 0], :, 0], want[table[2, 0], :, 1] = k[4], k[5]
    want[table[1, 0], :, 0] = k[3]        # position 1 - 2 + 1 = 0
    p = int(bad_sl[3]) - 2
    want[table[3, p // 16], :, p % 16] = k[6]
    assert torch.equal(kp.cpu(), want)


def test_append_far_page_offsets():
    """A pool of more than 2^31 elements: rows in its last page."""
    Hkv, d, ps = 8, 128, 64
    pages = 33000  # 33000 * 65536 elements > 2^31
    kp = torch.empty(pages, Hkv, ps, d, dtype=torch.bfloat16, device=DEV)
    vp = torch.empty_like(kp)
    k, v = (torch.randn(3, Hkv, d, device=DEV).to(torch.bfloat16) for _ in range(2))
    table = torch.tensor([[pages - 1], [pages - 2]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1, 3], dtype=torch.int32, device=DEV)
    sl = torch.tensor([ps, 2], dtype=torch.int32, device=DEV)
    ops.cache_append(k, v, kp, vp, table, cu, sl)
    assert ops.get_error() == ops.FA_OK
    assert torch.equal(kp[pages - 1, :, ps - 1], k[0]) and torch.equal(vp[pages - 2, :, :2], v[1:].transpose(0, 1))


def test_rope_refusals():
    q = torch.zeros(4, 2, 128, device=DEV, dtype=torch.bfloat16)
    pos = torch.zeros(4, device=DEV, dtype=torch.int32)
    inv = torch.ones(64, device=DEV)
    with pytest.raises(ValueError):
        ops.rope(q.half(), None, pos, inv)
    with pytest.raises(ValueError):
        ops.rope(q.transpose(0, 1), None, pos, inv)          # heads not contiguous
    with pytest.raises(ValueError):
        ops.rope(q, None, pos[:3], inv)                      # positions of fewer tokens
    with pytest.raises(ValueError):
        ops.rope(q, None, torch.zeros(2, 4, device=DEV, dtype=torch.int32), inv)  # axes missing
    with pytest.raises(ValueError):
        ops.rope(q, q.float(), pos, inv)                     # one type for both
    with pytest.raises(ops.FAError) as e:
        ops.rope(q, None, pos, torch.ones(65, device=DEV))   # more frequencies than pairs
    assert e.value.status == ops.FA_ERR_INVALID
    odd = torch.zeros(4, 2 * 128 + 4, device=DEV, dtype=torch.bfloat16)[:, :256].unflatten(1, (2, 128))
    with pytest.raises(ops.FAError) as e:
        ops.rope(odd, None, pos, inv)                        # rows not 16-byte aligned
    assert e.value.status == ops.FA_ERR_UNSUPPORTED
