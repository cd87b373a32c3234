"""E4M3 pages with scales at the ends of fp32's range, whose reciprocals are infinite or subnormal in
fp32.  The quotients here are formed in 64 bits; the scales and values are such that they keep well
away from the middle between two E4M3 numbers or are numbers of E4M3 themselves, so one byte is right."""
import pytest
import torch

from exact_io_aware_81_b200 import ops
from oracle import serving

pytestmark = pytest.mark.gpu

DEV = "cuda"


def append(values, scales, rotated):
    """One token, a K/V head per scale: `values` (128,) bf16 in every head -> bytes (heads, 128)."""
    H = len(scales)
    x = values.to(torch.bfloat16).view(1, 1, 128).expand(1, H, 128).contiguous().to(DEV)
    kp, vp = (torch.full((1, H, 16, 128), 0x55, dtype=torch.uint8, device=DEV) for _ in range(2))
    sc = torch.tensor(scales, dtype=torch.float64).float().to(DEV)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=DEV)  # noqa: E731
    where = kp, vp, i32([[0]]), i32([0, 1]), i32([1])
    if rotated:  # by an angle of 0: the same values, through the rotating kernels
        ops.rope_append(None, x, x, i32([0]), torch.ones(rotated, device=DEV), *where, k_scale=sc, v_scale=sc)
    else:
        ops.cache_append(x, x, *where, k_scale=sc, v_scale=sc)
    assert ops.get_error() == ops.FA_OK
    # the keys are the values, but for the sign of a zero, which x sin 0 + y cos 0 = 0 + (-0) = 0 loses
    assert torch.equal(torch.where(kp & 0x7F == 0, 0, kp), torch.where(vp & 0x7F == 0, 0, vp))
    assert (kp[:, :, 1:] == 0x55).all() and (vp[:, :, 1:] == 0x55).all()
    return kp[0, :, 0].cpu(), sc.cpu().double()


SCALES = [2.0 ** -149, 2.0 ** -148 * 1.5, 2.0 ** -130, 2.0 ** -129, 2.0 ** -128, 2.0 ** -127, 2.0 ** -126, 2.0 ** -100, 1.0, 2.0 ** 100,
          2.0 ** 126, 2.0 ** 126 * 1.75, 2.0 ** 127, 2.0 ** 127 * 1.875]


@pytest.mark.parametrize("rotated", [0, 64, 13])
@pytest.mark.parametrize("e", [-133, -126, -100, 0, 100, 117, 126])
def test_scales_at_the_ends_of_the_range(e, rotated):
    """Values of about 2^e, zeros of both signs among them."""
    m = torch.tensor([0.0, -0.0, 1.0, -1.0, 1.25, 1.5, -1.75, 0.5], dtype=torch.float64)
    x = (m * 2.0 ** e).repeat(16).float().to(torch.bfloat16)
    got, sc = append(x, SCALES, rotated)
    for h, s in enumerate(sc):
        want = serving.e4m3_bytes((x.double() / s).clamp(-1e30, 1e30).float())
        assert torch.equal(got[h] & 0x7F, want & 0x7F), f"scale {float(s)}"
        big = (want & 0x7F) != 0
        assert torch.equal(got[h][big], want[big])


@pytest.mark.parametrize("rotated", [0, 64, 13])
def test_values_that_are_not_finite_and_a_scale_of_zero(rotated):
    """As a division: NaN stays NaN, infinities saturate, 0 / 0 is NaN, x / 0 saturates."""
    x = torch.zeros(128)
    x[:6] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0, -1.0, 0.0])
    if rotated:
        x[:3] = 1.0   # (a pair with an infinity turns into NaN: that is the rotation's)
    got, _ = append(x, [0.0, 2.0 ** -149, 2.0 ** 127], rotated)
    for h in range(3):
        if not rotated:
            assert got[h][0] & 0x7F == 0x7F and got[h][1] == 0x7E and got[h][2] == 0xFE
    assert got[0][3] == 0x7E and got[0][4] == 0xFE and got[0][5] & 0x7F == 0x7F
    assert got[1][3] == 0x7E and got[1][4] == 0xFE and got[1][5] & 0x7F == 0
    assert (got[2][3:6] & 0x7F == 0).all()
