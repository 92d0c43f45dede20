"""RMS norm of rows that are not finite, or whose squares are not, at widths of each kernel."""
import math

import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build
from test_rms_norm import BF, F32, MODES, check_forward, forward, inputs

pytestmark = pytest.mark.gpu
# in registers (8, 16 and 32 columns a thread by the number of rows), through shared memory, long
WIDTHS = [40, 1000, 1001, 2050, 7167, 7168, 9000, 16384, 9001, 16400]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


@pytest.mark.parametrize("T", [7, 400])
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("mode", ["row", "block", "mx"])
def test_scales_of_rows_that_are_not_finite(T, H, dt, mode):
    """NaN does not enter the scales: a row of NaN has those of a row of zeros, and so has one with an infinity, whose
    rstd is zero."""
    x, _, gamma = inputs(T, H, dt)
    x[1, 5] = math.nan
    x[2] = math.nan
    x[3, H - 1] = math.inf
    x[4, 7], x[4, 9] = -math.inf, math.inf
    _, y, q, s, rstd = forward(x, None, gamma, mode)
    s, q = s.view(T, -1), q.float()
    assert bool((s[1:5] == (0 if mode == "mx" else 1)).all())
    assert bool(torch.isnan(q[1:3]).all()) and bool(torch.isnan(y[1:3]).all()) and not rstd[3:5].any()
    for row, at in ((3, [H - 1]), (4, [7, 9])):
        rest = torch.ones(H, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert bool(torch.isnan(q[row, at]).all()) and bool(torch.isnan(y[row, at]).all())
        assert not q[row, rest].any() and not y[row, rest].any()
    keep = [0] + list(range(5, T))
    pick = lambda v: v[keep].contiguous()       # noqa: E731
    check_forward(pick(x), None, gamma, (None, pick(y), pick(q), pick(s), pick(rstd)), mode)


@pytest.mark.parametrize("T", [7, 400])
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("mode", MODES)
def test_finite_rows_whose_squares_are_not(T, H, dt, mode):
    """rstd is 0, and y with it, however large gamma is beside h (an infinity, of BF16 here, times 0 is NaN)."""
    x, _, gamma = inputs(T, H, dt)
    gamma = gamma.abs() + 0.5
    x[1] = 3e38
    x[2, ::2] *= 2e38
    x[3, 3] = -3e38
    _, y, q, s, rstd = forward(x, None, gamma, mode)
    want = torch.where(x[1:4].isfinite(), 0.0, math.nan)
    same = lambda v: bool(((v == want) | (v.isnan() & want.isnan())).all())     # noqa: E731
    assert bool(x[1].isfinite().all()) and bool(x[3].isfinite().all())
    assert not rstd[1:4].any() and same(y[1:4].float())
    if mode is not None:
        assert same(q.float()[1:4]) and bool((s.view(T, -1)[1:4] == (0 if mode == "mx" else 1)).all())
    keep = [0] + list(range(4, T))
    pick = lambda v: None if v is None else v[keep].contiguous()       # noqa: E731
    check_forward(pick(x), None, gamma, (None, pick(y), pick(q), pick(s), pick(rstd)), mode)


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("mode", [None, "block", "mx"])
def test_large_gamma(H, dt, mode):
    """h gamma passes FP32, y does not."""
    x, _, gamma = inputs(9, H, dt, scale=1e17)
    gamma = gamma * 1e22
    check_forward(x, None, gamma, forward(x, None, gamma, mode), mode)


def whole(T, H, dt, seed=0):
    """Rows of whole numbers, whose squares add up exactly in any order."""
    g = torch.Generator("cuda").manual_seed(seed + H)
    x = torch.randint(-3, 4, (T, H), generator=g, device="cuda")
    return x.to(dt), 0.1 + torch.rand(H, generator=g, device="cuda")


@pytest.mark.parametrize("T", [5, 330])
@pytest.mark.parametrize("H", WIDTHS)
def test_one_rounding(T, H):
    """Where the sum of squares is exact, y is rounded once: half a unit, and the 2^-30 of rstd and h rstd in two numbers."""
    x, gamma = whole(T, H, F32)
    _, y, _, _, rstd = forward(x, None, gamma)
    r = (x.double().square().mean(1) + 1e-6).rsqrt()
    want = x.double() * r[:, None] * gamma.double()
    assert bool(((y.double() - want).abs() <= (2.0 ** -24 + 2.0 ** -30) * want.abs()).all())
    assert bool(((rstd.double() - r).abs() <= (2.0 ** -24 + 2.0 ** -30) * r).all())


@pytest.mark.parametrize("T", [5, 330])
@pytest.mark.parametrize("H", [8200, 12288, 16384])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("mode", MODES)
def test_a_row_at_an_odd_offset(T, H, dt, mode):
    """The kernel of rows off their vectors gives the same y, codes and scales where the sum is exact."""
    x, gamma = whole(T, H, dt)
    buf = torch.zeros(T, H + 5, dtype=dt, device="cuda")
    buf[:, 3:3 + H] = x
    a, b = forward(x, None, gamma, mode), forward(buf[:, 3:3 + H], None, gamma, mode)
    for u, v in zip(a[1:], b[1:]):
        assert u is None or torch.equal(u.view(torch.uint8), v.view(torch.uint8))


@pytest.mark.parametrize("T", [3, 200, 400])
@pytest.mark.parametrize("H", [8, 33, 100, 500, 1000, 1001, 1032, 2050, 4100, 7168, 8200, 9001, 16384, 16400])
@pytest.mark.parametrize("dt", [BF, F32])
def test_y_with_codes_and_without(T, H, dt):
    """The same y: BF16 rows, and FP32 rows of whole 16-byte blocks."""
    if dt == F32 and H % 4:
        H += 4 - H % 4
    x, res, gamma = inputs(T, H, dt)
    plain = forward(x, res, gamma)
    for mode in MODES[1:]:
        got = forward(x, res, gamma, mode)
        assert torch.equal(got[1], plain[1]) and torch.equal(got[0], plain[0]) and torch.equal(got[4], plain[4])
