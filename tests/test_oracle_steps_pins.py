"""The float64 formulas of layer norm, rotary positions and the expert permutation (oracle/steps.py), CPU only: against
torch's own layer norm and float64 autograd, closed forms, and the properties that fix them."""
import math

import numpy as np
import pytest
import torch

from oracle import steps

TIGHT = 1e-12  # float64 sums of a few hundred terms of order 1


def t64(*shape, seed=0):
    return torch.randn(*shape, dtype=torch.float64, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("hidden", [1, 2, 8, 300])
def test_layer_norm_and_its_gradients(hidden):
    x, dy, g, b = (t64(7, hidden, seed=1) + 0.4).requires_grad_(), t64(7, hidden, seed=2), t64(hidden, seed=3), t64(hidden, seed=4)
    gain, bias = (g - 1.0).requires_grad_(), b.clone().requires_grad_()
    y = torch.nn.functional.layer_norm(x, (hidden,), gain + 1.0, bias, 1e-3)
    y.backward(dy)
    n = [t.detach().numpy() for t in (x, dy, gain, bias)]
    got, mag = steps.layer_norm(n[0], n[2], n[3], 1.0, 1e-3)
    assert np.abs(got - y.detach().numpy()).max() < TIGHT and (mag >= np.abs(got) - TIGHT).all()
    for (d, m), want in zip(steps.layer_norm_bwd(n[0], n[1], n[2], 1.0, 1e-3), (x.grad, gain.grad, bias.grad)):
        assert np.abs(d - want.numpy()).max() < 1e-9 and (m >= np.abs(d) - TIGHT).all()


def test_layer_norm_closed_forms():
    x = np.array([[1.0, 3.0], [5.0, 5.0]])
    assert np.allclose(steps.layer_norm(x, eps=0.0 + 1e-30)[0][0], [-1.0, 1.0], atol=TIGHT)  # mean 2, variance 1
    assert not steps.layer_norm(x, eps=1e-6)[0][1].any()  # a constant row
    y = steps.layer_norm(t64(5, 64).numpy() * 3 + 7, eps=1e-9)[0]
    assert np.abs(y.mean(1)).max() < TIGHT and np.abs((y * y).mean(1) - 1).max() < 1e-8
    # the input gradient is orthogonal to the ones and (eps 0) to the normalised row
    x, dy = t64(5, 64, seed=1).numpy(), t64(5, 64, seed=2).numpy()
    dx = steps.layer_norm_bwd(x, dy, eps=1e-30)[0][0]
    assert np.abs(dx.sum(1)).max() < TIGHT and np.abs((dx * steps.layer_norm(x, eps=1e-30)[0]).sum(1)).max() < 1e-11


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
def test_rope(pairing):
    f = np.array([1.0, 0.25, 0.01])
    x = t64(4, 2, 8, seed=3).numpy()
    at0, _ = steps.rope(x, np.zeros(4), f, pairing)
    assert np.array_equal(at0, x)  # position 0 is the identity
    pos = np.array([3, 1, -2, 1000])
    y, mag = steps.rope(x, pos, f, pairing, 0.5)
    assert np.array_equal(y[..., 6:], x[..., 6:]) and not mag[..., 6:].any()  # what is not rotated
    for t in range(4):
        for i, w in enumerate(f):
            a, b = (i, i + 3) if pairing == "half" else (2 * i, 2 * i + 1)
            r = 0.5 * np.array([[math.cos(pos[t] * w), -math.sin(pos[t] * w)], [math.sin(pos[t] * w), math.cos(pos[t] * w)]])
            assert np.allclose(y[t][:, [a, b]], x[t][:, [a, b]] @ r.T, atol=1e-12)
    # the gradient is the transpose, and turns back
    u = t64(4, 2, 8, seed=4).numpy()
    assert abs((y * u).sum() - (x * steps.rope(u, pos, f, pairing, 0.5, backward=True)[0]).sum()) < 1e-11
    assert np.allclose(steps.rope(steps.rope(x, pos, f, pairing)[0], pos, f, pairing, backward=True)[0], x, atol=1e-12)
    # products of a query and a key depend on the distance alone
    q, k = t64(1, 1, 6, seed=5).numpy(), t64(1, 1, 6, seed=6).numpy()

    def product(m, n):
        return (steps.rope(q, [m], f, pairing)[0] * steps.rope(k, [n], f, pairing)[0]).sum()

    assert abs(product(7, 2) - product(100007, 100002)) < 1e-9


def test_rope_positions():
    assert list(steps.rope_positions(5, seqlen=2)) == [0, 1, 0, 1, 0]
    assert list(steps.rope_positions(5, cu_seqlens=[0, 0, 3, 3, 5])) == [0, 1, 2, 0, 1]


def test_rope_frequencies():
    none = steps.rope_frequencies(8, 16.0)
    assert np.allclose(none, [1.0, 0.5, 0.25, 0.125], atol=1e-15)
    assert np.allclose(steps.rope_frequencies(8, 16.0, "linear", 4.0), none / 4)
    base = steps.rope_frequencies(8, 16.0, "base", 4.0)
    assert base[0] == 1.0 and np.isclose(base[-1], none[-1] / 4)  # the last pair is stretched by the factor
    assert steps.rope_frequencies(2, 16.0, "base", 4.0)[0] == 1.0
    ctx = 2 * math.pi * 8  # pair i turns 8 f_i times
    bands = steps.rope_frequencies(8, 16.0, "bands", 4.0, 1.5, 3.0, ctx)
    assert np.allclose(bands, [1.0, 0.5, 0.25 * (1 / 3 + 2 / 3 / 4), 0.125 / 4])  # 8, 4, 2 and 1 turns
    ramp = steps.rope_frequencies(8, 16.0, "ramp", 4.0, 1.0, 4.0, ctx)  # pair 1 turns 4 times, pair 3 once
    assert np.allclose(ramp, [1.0, 0.5, 0.25 * (0.5 + 0.5 / 4), 0.125 / 4])


@pytest.mark.parametrize("tokens,top_k,experts", [(1, 1, 1), (50, 3, 7), (900, 4, 6)])
def test_experts(tokens, top_k, experts):
    ids = torch.randint(-1, experts + 1, (tokens, top_k), generator=torch.Generator().manual_seed(tokens)).numpy()
    off, row, slot = steps.expert_sort(ids, experts)
    kept = off[-1]
    flat = ids.reshape(-1)
    good = (flat >= 0) & (flat < experts)
    assert kept == good.sum() and off[0] == 0 and (np.diff(off) == np.bincount(flat[good], minlength=experts)).all()
    want = np.argsort(np.where(good, flat, experts), kind="stable")[:kept]
    assert np.array_equal(slot[:kept], want) and (slot[kept:] == -1).all()
    assert np.array_equal(row.reshape(-1)[want], np.arange(kept)) and (row.reshape(-1)[~good] == -1).all()
    # the gradients by autograd of the sums written with indices
    rows, w = t64(tokens * top_k, 5, seed=1).requires_grad_(), t64(tokens, top_k, seed=2).requires_grad_()
    at = torch.from_numpy(row.clip(0))
    y = (rows[at] * (w * torch.from_numpy(row >= 0))[..., None]).sum(1)
    dy = t64(tokens, 5, seed=3)
    y.backward(dy)
    got, mag = steps.expert_combine(rows.detach().numpy(), row, w.detach().numpy())
    assert np.abs(got - y.detach().numpy()).max() < TIGHT and (mag >= np.abs(got) - TIGHT).all()
    (drows, _), (dw, _) = steps.expert_combine_bwd(rows.detach().numpy(), dy.numpy(), row, w.detach().numpy())
    assert np.isnan(drows[kept:]).all() and np.abs(drows[:kept] - rows.grad.numpy()[:kept]).max(initial=0.0) < TIGHT
    assert np.abs(dw - w.grad.numpy()).max() < TIGHT
