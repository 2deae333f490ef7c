"""Layer norm and its backward on the GPU against the float64 formulas.

Units of 2^-24 (tests/close64.py), counted along an output's evaluation.  A row sum of H <= 32768 elements: at most 32
sums in a row inside a thread (4 slots of 8 elements; 8 of 8 in the widest rows, in two chains), 5 + 4 in the two
butterflies: 41, and one for 1 / H and its product each: 43.  Forward: the mean's error reaches the centred element once
(43 units of mean|x|); the variance carries 43 + 3 for its squares, halved by the root, + 2 ulp = 4 units of rsqrtf and
2 for the products, sum and gain, on the centred element: 23 + 6.  43 + 29 -> 80 units of mag cover both parts.
Backward: two rounds of such sums, r cubed (3 (23 + 4)) and four products: 43 + 43 + 81 + 8 -> 192.  Parameter
gradients add up rows: at most 8 in a row in a CTA at these sizes, 32 runs of the partials, 19 in one, 5 of the tree,
on top of n's 80: 128 + 64 -> 192.
"""
import numpy as np
import pytest
import torch

from gate_cores_b200 import _lib, cores
from oracle import steps

from .close64 import f64, near, same_bits

pytestmark = pytest.mark.gpu

FWD, BWD, PARAM = 80, 192, 192
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rows_of(rows, hidden, dt, seed=0, mean=0.0, spread=1.0):
    g = torch.Generator().manual_seed(seed + 1000 * rows + hidden)
    return (torch.randn(rows, hidden, generator=g) * spread + mean).to(dt).cuda()


def params(hidden, seed=0):
    g = torch.Generator().manual_seed(seed + hidden)
    return (0.5 + torch.rand(hidden, generator=g)).cuda(), torch.randn(hidden, generator=g).cuda()


# one row, odd row counts, one vector, odd vector counts, each number of slots per thread, the widest rows
SHAPES = [(1, 8), (1, 512), (3, 40), (37, 264), (1, 1000), (5, 1280), (129, 2056), (9, 2304), (11, 2600), (10, 3328), (700, 4096), (33, 5120),
          (9, 6144), (12, 7168), (61, 8192)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,hidden", SHAPES + [(3, 9000), (4, 12544), (7, 13824), (2, 16384)])
@pytest.mark.parametrize("which", ["gain_bias", "plain", "bias", "zero_centered"])
def test_forward(cuda_ok, dt, rows, hidden, which):
    x = rows_of(rows, hidden, DT[dt], mean=0.3)
    g, b = params(hidden)
    gain, bias, off = {"gain_bias": (g, b, 0.0), "plain": (None, None, 0.0), "bias": (None, b, 0.0),
                       "zero_centered": (g - 1.0, None, 1.0)}[which]
    y = cores.layer_norm(x, gain, bias, off, eps=1e-5)
    ref = steps.layer_norm(f64(x), None if gain is None else f64(gain), None if bias is None else f64(bias), off,
                           float(np.float32(1e-5)))
    near(y, ref, FWD, f"{dt} {rows}x{hidden} {which}")
    assert _lib.muse_device_error() == 0


def test_forward_widest_bf16(cuda_ok):
    x = rows_of(5, 32768, torch.bfloat16)
    g, b = params(32768)
    near(cores.layer_norm(x, g, b), steps.layer_norm(f64(x), f64(g), f64(b), 0.0, float(np.float32(1e-6))), FWD)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hidden", [264, 4096, 16384])
def test_forward_mean_far_from_zero(cuda_ok, dt, hidden):
    # the variance of elements 300 spreads away from zero, and constant rows (variance 0: y is the bias, to the mean's rounding)
    x = rows_of(9, hidden, DT[dt], mean=300.0)
    x[4] = 7.25
    x[5] = 0.0
    g, b = params(hidden)
    y = cores.layer_norm(x, g, b)
    near(y, steps.layer_norm(f64(x), f64(g), f64(b), 0.0, float(np.float32(1e-6))), FWD)
    assert torch.equal(y[5], b.to(DT[dt]))
    if dt == "f32":
        # FP32 rows: the elements' differences from the mean are exact (both within a factor of two), so that what is
        # rounded has the spread's size and not the mean's
        c = f64(x) - f64(x).mean(-1, keepdims=True)
        r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + float(np.float32(1e-6)))
        mag = (np.abs(c) + np.abs(c).mean(-1, keepdims=True)) * r * f64(g) + np.abs(f64(b))
        spread = np.arange(9) != 4
        near(y[torch.from_numpy(spread)], ((c * r * f64(g) + f64(b))[spread], mag[spread]), FWD)


@pytest.mark.parametrize("hidden", [264, 4096])
def test_forward_outliers(cuda_ok, hidden):
    x = rows_of(17, hidden, torch.bfloat16)
    x[:, ::100] *= 1000
    g, b = params(hidden)
    near(cores.layer_norm(x, g, b), steps.layer_norm(f64(x), f64(g), f64(b), 0.0, float(np.float32(1e-6))), FWD)


def test_a_row_with_nan_or_inf_leaves_the_others(cuda_ok):
    x = rows_of(200, 4096, torch.bfloat16)
    g, b = params(4096)
    clean = cores.layer_norm(x, g, b)
    x[3, 77], x[150, 0] = float("nan"), float("inf")
    y = cores.layer_norm(x, g, b)
    keep = torch.ones(200, dtype=torch.bool)
    keep[[3, 150]] = False
    assert same_bits(y[keep], clean[keep])
    assert torch.isnan(y[3]).all() and torch.isnan(y[150]).all()


@pytest.mark.parametrize("dt", DT)
def test_strides_in_place_and_three_dims(cuda_ok, dt):
    wide = rows_of(50, 1024, DT[dt])
    g, b = params(512)
    view = wide[:, 256:768]
    want = cores.layer_norm(view.contiguous(), g, b)
    into = torch.full((50, 1024), 3.0, dtype=DT[dt], device="cuda")
    cores.layer_norm(view, g, b, out=into[:, 512:])
    assert same_bits(into[:, 512:], want) and bool((into[:, :512] == 3.0).all())
    assert same_bits(cores.layer_norm(view.contiguous().view(5, 10, 512), g, b).view(50, 512), want)
    rest = wide.clone()
    cores.layer_norm(view, g, b, out=view)
    assert same_bits(view, want) and same_bits(wide[:, :256], rest[:, :256]) and same_bits(wide[:, 768:], rest[:, 768:])


def test_no_rows(cuda_ok):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    g, b = params(64)
    assert cores.layer_norm(x, g, b).shape == (0, 64)
    dx, dg, db = cores.layer_norm_backward(x, x, g)
    assert dx.shape == (0, 64) and not dg.any() and not db.any()


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("which", ["gain", "plain", "zero_centered"])
def test_backward(cuda_ok, dt, rows, hidden, which):
    if dt == "f32" and hidden > 4096:
        pytest.skip("FP32 backward rows are limited to 4096 elements")
    x, dy = rows_of(rows, hidden, DT[dt], mean=0.3), rows_of(rows, hidden, DT[dt], seed=5)
    g, _ = params(hidden)
    gain, off = {"gain": (g, 0.0), "plain": (None, 0.0), "zero_centered": (g - 1.0, 1.0)}[which]
    dx, dg, db = cores.layer_norm_backward(x, dy, gain, off, eps=1e-5)
    rx, rg, rb = steps.layer_norm_bwd(f64(x), f64(dy), None if gain is None else f64(gain), off, float(np.float32(1e-5)))
    near(dx, rx, BWD, "dx")
    near(db, rb, PARAM, "dbias")
    assert (dg is None) == (gain is None)
    if gain is not None:
        near(dg, rg, PARAM, "dgain")
    assert _lib.muse_device_error() == 0


@pytest.mark.parametrize("dt", DT)
def test_backward_mean_far_from_zero(cuda_ok, dt):
    x, dy = rows_of(40, 1000, DT[dt], mean=300.0), rows_of(40, 1000, DT[dt], seed=5)
    x[7] = -3.5  # a constant row: n is 0, r is 1 / sqrt(eps)
    g, _ = params(1000)
    got = cores.layer_norm_backward(x, dy, g, eps=1e-3)
    for t, ref, u in zip(got, steps.layer_norm_bwd(f64(x), f64(dy), f64(g), 0.0, float(np.float32(1e-3))), (BWD, PARAM, PARAM)):
        near(t, ref, u)


def test_backward_against_differences(cuda_ok):
    # d/dx of sum(y * u) by central differences of the float64 formula, at a few places
    x, u = rows_of(4, 64, torch.float32), rows_of(4, 64, torch.float32, seed=3)
    g, b = params(64)
    dx, dg, db = (f64(t) for t in cores.layer_norm_backward(x, u, g, eps=1e-5))
    eps, h = float(np.float32(1e-5)), 1e-5

    def loss(x_, g_, b_):
        return float((steps.layer_norm(x_, g_, b_, 0.0, eps)[0] * f64(u)).sum())

    for i, j in [(0, 0), (1, 17), (3, 63)]:
        e = np.zeros((4, 64))
        e[i, j] = h
        # the differences' own error is below 1e-8 (h^2 times third derivatives of order 1; 2^-52 of a loss of order 100
        # over h); the kernel's is BWD units of 2^-24 of a mag of at most 8: 1e-4
        assert abs((loss(f64(x) + e, f64(g), f64(b)) - loss(f64(x) - e, f64(g), f64(b))) / (2 * h) - dx[i, j]) < 1e-4
        v = np.zeros(64)
        v[j] = h
        assert abs((loss(f64(x), f64(g) + v, f64(b)) - loss(f64(x), f64(g) - v, f64(b))) / (2 * h) - dg[j]) < 1e-4
        assert abs((loss(f64(x), f64(g), f64(b) + v) - loss(f64(x), f64(g), f64(b) - v)) / (2 * h) - db[j]) < 1e-4


@pytest.mark.parametrize("alias", ["x", "dy"])
def test_backward_in_place_and_parts(cuda_ok, alias):
    x, dy = rows_of(300, 2048, torch.bfloat16), rows_of(300, 2048, torch.bfloat16, seed=2)
    g, _ = params(2048)
    want = cores.layer_norm_backward(x, dy, g)
    again = cores.layer_norm_backward(x, dy, g)
    assert all(same_bits(a, b) for a, b in zip(want, again))  # the same bits every time
    only_dx = cores.layer_norm_backward(x, dy, g, want_dgain=False, want_dbias=False)
    assert same_bits(only_dx[0], want[0]) and only_dx[1] is None and only_dx[2] is None
    assert same_bits(cores.layer_norm_backward(x, dy, g, want_dgain=False)[2], want[2])
    assert same_bits(cores.layer_norm_backward(x, dy, g, want_dbias=False)[1], want[1])
    x2, dy2 = x.clone(), dy.clone()
    got = cores.layer_norm_backward(x2, dy2, g, dx=x2 if alias == "x" else dy2)
    assert all(same_bits(a, b) for a, b in zip(want, got))


def test_backward_strided_and_own_workspace(cuda_ok):
    wide = rows_of(77, 1600, torch.float32)
    x, dy = wide[:, :520], wide[:, 800:1320]
    g, _ = params(520)
    want = cores.layer_norm_backward(x.contiguous(), dy.contiguous(), g)
    ws = torch.full((_lib.muse_norm_backward_workspace_bytes(77, 520),), 255, dtype=torch.uint8, device="cuda")
    got = cores.layer_norm_backward(x, dy, g, workspace=ws)
    assert all(same_bits(a, b) for a, b in zip(want, got))


def test_another_stream_and_a_graph(cuda_ok):
    x, dy = rows_of(500, 1280, torch.bfloat16), rows_of(500, 1280, torch.bfloat16, seed=2)
    g, b = params(1280)
    want = (cores.layer_norm(x, g, b),) + cores.layer_norm_backward(x, dy, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (cores.layer_norm(x, g, b, stream=side),) + cores.layer_norm_backward(x, dy, g, stream=side.cuda_stream)
    side.synchronize()
    assert all(same_bits(a, c) for a, c in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = (cores.layer_norm(x, g, b),) + cores.layer_norm_backward(x, dy, g)
    x.copy_(x.flip(0))
    dy.copy_(dy.flip(0))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert same_bits(held[0], want[0].flip(0)) and same_bits(held[1], want[1].flip(0))
    rx, rg, rb = steps.layer_norm_bwd(f64(x), f64(dy), f64(g), 0.0, float(np.float32(1e-6)))
    near(held[2], rg, PARAM)
    near(held[3], rb, PARAM)


def test_refusals(cuda_ok):
    x = rows_of(4, 64, torch.bfloat16)
    g, b = params(64)
    for bad in (lambda: cores.layer_norm(x, g[:32], b), lambda: cores.layer_norm(x, g, b[None].expand(2, 64)),
                lambda: cores.layer_norm(x.T, None, None), lambda: cores.layer_norm(x, out=x[:2]),
                lambda: cores.layer_norm(x, g.cpu()), lambda: cores.layer_norm_backward(x, x[:2]),
                lambda: cores.layer_norm_backward(x, x.float())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cores.layer_norm(x, g.double()), lambda: cores.layer_norm(x.half())):
        with pytest.raises(TypeError):
            bad()
    for bad, status in ((lambda: cores.layer_norm(rows_of(4, 60, torch.bfloat16)), _lib.MUSE_ERR_UNSUPPORTED),
                        (lambda: cores.layer_norm(x[:1].expand(4, 64)), _lib.MUSE_ERR_INVALID_ARGUMENT),
                        (lambda: cores.layer_norm(x, eps=-1.0), _lib.MUSE_ERR_INVALID_ARGUMENT)):
        with pytest.raises(_lib.MuseError) as e:
            bad()
        assert e.value.status == status


def test_a_workspace_that_is_not_its_own_bytes(cuda_ok):
    x, dy = rows_of(9, 64, torch.float32), rows_of(9, 64, torch.float32, seed=1)
    need = _lib.muse_norm_backward_workspace_bytes(9, 64)
    whole = torch.empty(2 * need, dtype=torch.uint8, device="cuda")
    for ws in (whole[:1].expand(need), whole[::2], whole[:need - 1]):
        with pytest.raises(ValueError):
            cores.layer_norm_backward(x, dy, workspace=ws)
