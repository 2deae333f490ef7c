"""Layer norm of rows whose elements are all one value, or nearly: what the mean's rounding leaves must not be lifted by
1 / sqrt(eps).

With K = 43 units of 2^-24 for a sum over a row (test_gpu_layer_norm.py), an FP32 row's mean is off by at most K u
mean|x|.  The elements less that mean are exact or off by a unit of themselves, and their own mean, which is taken off as
well, by K u of the mean of their sizes, mean|x - m| + K u mean|x|.  So the magnitudes that are rounded are those of the
centred elements, and of mean|x| a part of 43 * 2^-24.

bf16 rows: the values below are multiples of one step of bf16 with 8 bits, or a step more, so sums of up to 2^15 of them
are exact in 24 bits.  The mean of a row of one value is that value then, and nothing is left.  Otherwise the mean is
rounded (a unit of itself, in each warp and where they are joined) and mean * r once more: 4 units of |mean| r.
"""
import numpy as np
import pytest
import torch

from gate_cores_b200 import cores

from .close64 import f64, near
from .test_gpu_layer_norm import BWD, DT, FWD, PARAM, params

pytestmark = pytest.mark.gpu

EPS = 1e-6
EPS64 = float(np.float32(EPS))
K = 43 * 2.0 ** -24
# powers of two and others, values whose sums round, and one that steps up by an element's last place
VALUES = [2576.0, 7.25, -3.328125, 0.33203125, 1.0, 300.0, -1e4, 0.0]
WIDTHS = [24, 264, 520, 1000, 1544, 2600, 4096, 7168]


def rows_of_values(rows, hidden, dt):
    v = torch.tensor(VALUES)[torch.arange(rows) % len(VALUES)]
    x = v[:, None].repeat(1, hidden).to(dt)
    odd = torch.arange(rows) % 3 == 1  # a third of the rows with one element that is one step of bf16 larger
    x[odd, (5 * torch.arange(rows) % hidden)[odd]] *= 1.0 + 2.0 ** -7
    return x.cuda()


def parts(x, dt, units):
    """(centred elements, r, off): n's error in units is `units` times off, beside n's own."""
    m = x.mean(-1, keepdims=True)
    c = x - m
    r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + EPS64)
    rounded = K * np.abs(x).mean(-1, keepdims=True)
    if dt == torch.bfloat16:
        rounded = 4 / units * np.abs(m) * (x != x[:, :1]).any(-1, keepdims=True)
    return c, r, r * (np.abs(c).mean(-1, keepdims=True) + rounded)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hidden", WIDTHS + [9000, 12296, 16000])
@pytest.mark.parametrize("rows", [11, 400])
def test_forward(cuda_ok, dt, hidden, rows):
    x = rows_of_values(rows, hidden, DT[dt])
    g, b = params(hidden)
    c, r, off = parts(f64(x), DT[dt], FWD)
    n, w = c * r, f64(g)
    mag = (np.abs(n) + off) * np.abs(w) + np.abs(f64(b))
    near(cores.layer_norm(x, g, b, eps=EPS), (n * w + f64(b), mag), FWD, f"{rows} x {hidden}")


def test_forward_widest_bf16(cuda_ok):
    x = rows_of_values(9, 32760, torch.bfloat16)
    c, r, off = parts(f64(x), torch.bfloat16, FWD)
    near(cores.layer_norm(x, eps=EPS), (c * r, np.abs(c * r) + off), FWD)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hidden", WIDTHS)
@pytest.mark.parametrize("rows", [11, 400])
def test_backward(cuda_ok, dt, hidden, rows):
    if dt == "f32" and hidden > 4096:
        pytest.skip("FP32 backward rows are limited to 4096 elements")
    x = rows_of_values(rows, hidden, DT[dt])
    gen = torch.Generator().manual_seed(rows + hidden)
    dy = torch.randn(rows, hidden, generator=gen).to(DT[dt]).cuda()
    gain, _ = params(hidden)
    c, r, off = parts(f64(x), DT[dt], PARAM)
    n, d = c * r, f64(dy)
    g = d * f64(gain)
    gm, gn = np.abs(g).mean(-1, keepdims=True), (g * n).mean(-1, keepdims=True)
    dx = r * (g - g.mean(-1, keepdims=True) - n * gn)
    mag = r * (np.abs(g) + gm + (np.abs(n) + off) * (np.abs(g * n).mean(-1, keepdims=True) + off * gm))
    got = cores.layer_norm_backward(x, dy, gain, eps=EPS)
    near(got[0], (dx, mag), BWD, "dx")
    near(got[1], ((d * n).sum(0), (np.abs(d) * (np.abs(n) + off)).sum(0)), PARAM, "dgain")
    near(got[2], (d.sum(0), np.abs(d).sum(0)), PARAM, "dbias")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hidden", WIDTHS)
@pytest.mark.parametrize("rows", [8, 403])
def test_rows_of_one_value_have_no_gain_gradient(cuda_ok, dt, hidden, rows):
    # n is 0 in all of them: bf16 rows give exactly that
    if dt == "f32" and hidden > 4096:
        pytest.skip("FP32 backward rows are limited to 4096 elements")
    x = torch.tensor(VALUES)[torch.arange(rows) % len(VALUES)][:, None].repeat(1, hidden).to(DT[dt]).cuda()
    gen = torch.Generator().manual_seed(rows + hidden)
    dy = torch.randn(rows, hidden, generator=gen).to(DT[dt]).cuda()
    gain, _ = params(hidden)
    c, r, off = parts(f64(x), DT[dt], PARAM)
    _, dgain, dbias = cores.layer_norm_backward(x, dy, gain, eps=EPS)
    near(dgain, (np.zeros(hidden), (np.abs(f64(dy)) * off).sum(0)), PARAM, "dgain")
    near(dbias, (f64(dy).sum(0), np.abs(f64(dy)).sum(0)), PARAM, "dbias")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hidden", [24, 264, 1000, 4096])
def test_squares_that_underflow(cuda_ok, dt, hidden):
    # elements of 1e-23: their squares sum to 0 in FP32, but they are not of one value; eps decides r
    gen = torch.Generator().manual_seed(hidden)
    x = (torch.randn(300, hidden, generator=gen) * 1e-23).to(DT[dt]).cuda()
    dy = torch.randn(300, hidden, generator=gen).to(DT[dt]).cuda()
    gain, _ = params(hidden)
    c, r, _ = parts(f64(x), DT[dt], PARAM)
    off = r * np.abs(f64(x)).mean(-1, keepdims=True)
    n, w, d = c * r, f64(gain), f64(dy)
    near(cores.layer_norm(x, gain, eps=EPS), (n * w, (np.abs(n) + off) * np.abs(w)), FWD)
    _, dgain, _ = cores.layer_norm_backward(x, dy, gain, eps=EPS)
    near(dgain, ((d * n).sum(0), (np.abs(d) * (np.abs(n) + off)).sum(0)), PARAM)


@pytest.mark.parametrize("dt", DT)
def test_rows_of_one_value_without_eps_are_nan(cuda_ok, dt):
    x = torch.full((9, 1000), 2576.0, dtype=DT[dt], device="cuda")
    x[0] = torch.randn(1000, device="cuda").to(DT[dt])
    gain, _ = params(1000)
    y = cores.layer_norm(x, gain, eps=0.0)
    assert torch.isfinite(y[0]).all()
    dx, dgain, dbias = cores.layer_norm_backward(x, x, gain, eps=0.0)
    assert torch.isfinite(dx[0]).all() and torch.isfinite(dbias).all()
    if dt == "bf16":  # (of an FP32 row the mean's rounding may be left, and that is not 0)
        assert torch.isnan(y[1:]).all() and torch.isnan(dgain).all()
