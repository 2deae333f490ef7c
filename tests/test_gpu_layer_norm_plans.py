"""Layer norm on the GPU in every way its launcher deals a row to lanes, with more rows than are on their way at a time.

The widths below reach, for each type, every number of lanes a row (4, 8, 16, 32 and whole warps) with every number of
vectors a lane that goes with it.  The row counts give a CTA at least three tiles even where an SM is full of them (2048
threads), so that places in shared memory are filled again, and leave the last tile partly empty.  The formulas are
evaluated in float64 on the GPU, with elementary operations.

Units of 2^-24 as in test_gpu_layer_norm.py.  Parameter gradients: every s-th row alone has a gradient (so that a row
lost, doubled or taken for another one is far above the tolerance), of which a CTA's thread adds at most 49 in a row
(`most_in_a_row`), then 32 runs of the partials, 19 in one, 5 of the tree, on top of n's 80: 185 <= 192.
"""
import pytest
import torch

from gate_cores_b200 import _lib, cores

from .close64 import HALF_STEP, same_bits
from .test_gpu_layer_norm import BWD, DT, FWD, PARAM

pytestmark = pytest.mark.gpu

EPS = 1e-5
EPS64 = float(torch.tensor(EPS, dtype=torch.float32))


def near64(got, want, mag, units, what):
    """tests/close64.py's rule, on the GPU."""
    off = units * 2.0 ** -24 * mag
    ok = (got.double() - want).abs() <= off + HALF_STEP[got.dtype] * (want.abs() + off)
    assert got.shape == want.shape
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()} off, first {(~ok).nonzero()[:4].tolist()}"


def normal(rows, hidden, dt, seed, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000 * rows + hidden)
    return (torch.randn(rows, hidden, generator=g, device="cuda") + mean).to(dt)


def vector(hidden, seed):
    return normal(1, hidden, torch.float32, seed)[0]


def norms(x, eps):
    x = x.double()
    m = x.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + eps)
    return (x - m) * r, r, x.abs().mean(-1, keepdim=True) * r


def forward64(x, gain, bias, eps):
    n, _, off = norms(x, eps)
    w = gain.double()
    return n * w + bias.double(), (n * w).abs() + off * w.abs() + bias.double().abs()


def backward64(x, dy, gain, eps):
    n, r, off = norms(x, eps)
    dy = dy.double()
    g = dy * gain.double()
    gm, gnm = g.abs().mean(-1, keepdim=True), (g * n).abs().mean(-1, keepdim=True)
    dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    return ((dx, r * (g.abs() + gm + (n.abs() + off) * (gnm + off * gm))),
            ((dy * n).sum(0), (dy.abs() * (n.abs() + off)).sum(0)), (dy.sum(0), dy.abs().sum(0)))


def lanes_of(hidden, dt, most):
    """Lanes of a row, `most` vectors each at most."""
    vectors = hidden // (8 if dt == torch.bfloat16 else 4)
    lanes = 4
    while lanes < 32 and lanes * most < vectors:
        lanes *= 2
    return lanes if lanes < 32 else 32 * (-(-vectors // (32 * most)))


def many_rows(lanes):
    """Rows that make three tiles a CTA and a part of one."""
    return 3 * 148 * 2048 // lanes + 17


FORWARD = {
    "bf16": [24, 56, 88, 120, 152, 184, 216, 248, 264, 376, 440, 504, 520, 712, 776, 1000, 1048, 1280, 1400, 1544, 1928, 2056, 2600,
             3328, 3848, 4104, 5120, 6024, 6400, 7168, 8192],
    "f32": [12, 28, 44, 60, 76, 92, 108, 124, 132, 188, 220, 252, 260, 356, 420, 500, 524, 640, 700, 772, 1000, 1048, 1300, 1700, 2000, 2056,
            2600, 2900, 3332, 4000, 4300, 4800, 5200, 6000, 6200, 7000, 8000],
}


@pytest.mark.parametrize("dt,hidden", [(d, h) for d in FORWARD for h in FORWARD[d]])
def test_forward_many_rows(cuda_ok, dt, hidden):
    rows = many_rows(lanes_of(hidden, DT[dt], 8))
    x, gain, bias = normal(rows, hidden, DT[dt], 1, 0.3), 1.0 + 0.3 * vector(hidden, 2), vector(hidden, 3)
    y = cores.layer_norm(x, gain, bias, eps=EPS)
    near64(y, *forward64(x, gain, bias, EPS64), FWD, f"{rows} x {hidden}")
    # in place: no row is read again once it is written
    assert same_bits(cores.layer_norm(x, gain, bias, eps=EPS, out=x), y)
    assert _lib.muse_device_error() == 0


# rows too wide for two on their way, or for the parameters in shared memory
@pytest.mark.parametrize("dt,hidden", [("bf16", 8200), ("bf16", 9000), ("bf16", 10504), ("bf16", 12400), ("bf16", 13000), ("bf16", 14000),
                                       ("bf16", 16384), ("bf16", 16392), ("bf16", 20000), ("f32", 8196), ("f32", 9500),
                                       ("f32", 12000), ("f32", 13900), ("f32", 14800), ("f32", 16384)])
def test_forward_wide_rows(cuda_ok, dt, hidden):
    rows = 148 * 4 * 3 + 5
    x, gain, bias = normal(rows, hidden, DT[dt], 1, 0.3), 1.0 + 0.3 * vector(hidden, 2), vector(hidden, 3)
    near64(cores.layer_norm(x, gain, bias, eps=EPS), *forward64(x, gain, bias, EPS64), FWD, f"{rows} x {hidden}")


# few rows: a row over as many warps as take it two vectors a lane
@pytest.mark.parametrize("dt,hidden", [("bf16", h) for h in (520, 1048, 1544, 2056, 2600, 3328, 4104, 4616, 5632, 6152, 6664, 7176, 8192)] +
                         [("f32", h) for h in (260, 516, 1000, 1284, 1540, 2052, 2600, 3076, 3332, 3588, 4096)])
@pytest.mark.parametrize("rows", [3, 296])
def test_forward_few_rows(cuda_ok, dt, hidden, rows):
    x, gain, bias = normal(rows, hidden, DT[dt], 1, 0.3), 1.0 + 0.3 * vector(hidden, 2), vector(hidden, 3)
    near64(cores.layer_norm(x, gain, bias, eps=EPS), *forward64(x, gain, bias, EPS64), FWD, f"{rows} x {hidden}")


# one width at least for each way to deal a row: lanes or warps of it, vectors a lane
BACKWARD = {
    "bf16": [24, 56, 88, 120, 160, 248, 264, 376, 504, 520, 600, 1000, 1048, 1800, 2056, 2600, 3600, 4104, 5128, 6152, 8192],
    "f32": [12, 24, 44, 60, 84, 116, 132, 160, 252, 260, 500, 600, 1000, 1100, 1500, 1700, 2000, 2100, 2500, 2600, 2900, 3332, 4000],
}


def most_in_a_row(rows, every, lanes):
    """Rows with a gradient that a thread adds: of each tile of its CTA's (192 threads' rows or more, one at least), one CTA of 148."""
    tile = max(1, 192 // lanes)
    return -(-rows // (tile * 148)) * -(-tile // every)


@pytest.mark.parametrize("dt,hidden", [(d, h) for d in BACKWARD for h in BACKWARD[d]])
def test_backward_many_rows(cuda_ok, dt, hidden):
    lanes = lanes_of(hidden, DT[dt], 4)
    rows = many_rows(lanes)
    x, gain = normal(rows, hidden, DT[dt], 1, 0.3), 1.0 + 0.3 * vector(hidden, 2)
    dense = normal(rows, hidden, DT[dt], 3)
    dx, _, _ = cores.layer_norm_backward(x, dense, gain, eps=EPS)
    near64(dx, *backward64(x, dense, gain, EPS64)[0], BWD, f"dx {rows} x {hidden}")
    every = rows // 2000 | 1
    assert most_in_a_row(rows, every, lanes) <= 49
    some = torch.zeros_like(dense)
    some[::every] = dense[::every]
    got = cores.layer_norm_backward(x, some, gain, eps=EPS)
    want = backward64(x, some, gain, EPS64)
    near64(got[1], *want[1], PARAM, f"dgain {rows} x {hidden}")
    near64(got[2], *want[2], PARAM, f"dbias {rows} x {hidden}")
    again = cores.layer_norm_backward(x, some, gain, eps=EPS, dx=x)
    assert all(same_bits(a, b) for a, b in zip(got, again))
    assert _lib.muse_device_error() == 0
