"""Rotary positions on the GPU against the float64 formulas (angles in extended precision).

Units of 2^-24 of mag = scale (|a| + |b|): cos and sin are off by at most 2 ulp of sincospif (2 units of a value up to
1), half a unit from the rounding of its argument (an eighth of a turn in 24 bits, times pi / 4 below 1) and 2^-33 turns
from the table's; the scale's product 1, the rotation's product and sum 1 each: 2 + 0.5 + 1 + 2 -> 8 with a margin.
"""
import numpy as np
import pytest
import torch

from gate_cores_b200 import _lib, cores
from oracle import steps

from .close64 import f64, near, same_bits

pytestmark = pytest.mark.gpu

UNITS = 8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def qk(tokens, hq, hk, d, dt, seed=0, fused=False):
    g = torch.Generator().manual_seed(seed + 131 * tokens + d)
    both = torch.randn(tokens, hq + 2 * hk, d, generator=g).to(dt).cuda()
    q, k = both[:, :hq], both[:, hq:hq + hk]
    return (q, k) if fused else (q.contiguous(), k.contiguous())


def check(x, got, positions, freq, pairing, scale=1.0, backward=False, what=""):
    tokens = x.numel() // (x.shape[-1] * x.shape[-2])
    ref = steps.rope(f64(x).reshape(tokens, *x.shape[-2:]), positions, f64(freq), pairing, scale, backward)
    near(got.reshape(tokens, *x.shape[-2:]), ref, UNITS, what)


# head_dim, rotary_dim: whole heads, parts, a part that ends inside a vector, halves that are no whole vectors, two elements
HEADS = [(128, 128), (128, 64), (64, 64), (80, 80), (80, 40), (80, 20), (96, 24), (256, 256), (40, 36), (16, 2), (8, 8)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("d,rd", HEADS)
@pytest.mark.parametrize("pairing", ["interleaved", "half"])
@pytest.mark.parametrize("backward", [False, True], ids=["fwd", "bwd"])
def test_heads(cuda_ok, dt, d, rd, pairing, backward):
    if dt == "f32" and d > 128:
        pytest.skip("FP32 heads are limited to 128 elements")
    call = cores.rope_backward if backward else cores.rope
    for tokens, hq, hk in ((1, 1, 1), (37, 5, 2), (300, 6, 6)):
        q, k = qk(tokens, hq, hk, d, DT[dt])
        f = cores.rope_frequencies(rd, 1e4)
        pos = (torch.arange(tokens, dtype=torch.int32) * 977 % 131072).cuda()
        qo, ko = call(q, k, f, positions=pos, pairing=pairing, attention_scale=1.25)
        for x, y in ((q, qo), (k, ko)):
            check(x, y, pos.cpu().numpy(), f, pairing, 1.25, backward, f"{tokens} tokens")
            assert same_bits(y[..., rd:], x[..., rd:])


@pytest.mark.parametrize("hq,hk", [(1, 0), (32, 8), (3, 5), (64, 1), (2, 64)])
def test_head_counts_and_q_alone(cuda_ok, hq, hk):
    q, k = qk(70, hq, max(hk, 1), 64, torch.bfloat16)
    f = cores.rope_frequencies(64, 5e5)
    qo, ko = cores.rope(q.view(2, 35, hq, 64), k.view(2, 35, hk, 64) if hk else None, f, pairing="half")
    pos = steps.rope_positions(70, 35)
    check(q, qo, pos, f, "half")
    if hk:
        check(k, ko, pos, f, "half")
    else:
        assert ko is None


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
def test_far_and_negative_positions(cuda_ok, pairing):
    pos = torch.tensor([0, 1, 131071, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -1, -(2 ** 31)], dtype=torch.int32).cuda()
    q, k = qk(8, 2, 1, 128, torch.float32)
    for f in (cores.rope_frequencies(128, 1e4), torch.rand(64, dtype=torch.float64).cuda() * 20 - 10):
        qo, ko = cores.rope(q, k, f, positions=pos, pairing=pairing)
        check(q, qo, pos.cpu().numpy(), f, pairing)
        check(k, ko, pos.cpu().numpy(), f, pairing)
        assert same_bits(qo[0], q[0])  # position 0 is the identity


@pytest.mark.parametrize("lengths", [[1], [5, 1, 64, 3], [0, 7, 0, 0, 20, 0], [1] * 100, [2000, 13]])
def test_packed_documents(cuda_ok, lengths):
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    tokens = int(cu[-1])
    q, k = qk(tokens, 4, 2, 128, torch.bfloat16)
    f = cores.rope_frequencies(128, 1e4)
    qo, ko = cores.rope(q, k, f, cu_seqlens=cu.cuda())
    pos = np.concatenate([np.arange(n) for n in lengths])
    check(q, qo, pos, f, "interleaved")
    check(k, ko, pos, f, "interleaved")


def test_boundaries_that_cover_too_few_tokens(cuda_ok):
    # tokens behind the last boundary: unspecified positions, but nothing is read or written out of bounds
    q, k = qk(50, 2, 1, 64, torch.bfloat16)
    qo, _ = cores.rope(q, k, cores.rope_frequencies(64), cu_seqlens=torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda"))
    check(q[:20], qo[:20], np.concatenate([np.arange(10)] * 2), cores.rope_frequencies(64), "interleaved")


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("d,rd,pairing", [(128, 128, "half"), (128, 64, "interleaved"), (80, 20, "half"), (96, 24, "interleaved"),
                                          (80, 36, "interleaved"), (128, 32, "half")])
def test_in_place_on_a_fused_projection(cuda_ok, dt, d, rd, pairing):
    q, k = qk(200, 6, 2, d, DT[dt], fused=True)
    whole = q._base if q._base is not None else q
    before = whole.clone()
    f = cores.rope_frequencies(rd)
    want = cores.rope(q, k, f, pairing=pairing)
    assert want[0].is_contiguous()
    got = cores.rope(q, k, f, pairing=pairing, q_out=q, k_out=k)
    assert same_bits(got[0], want[0]) and same_bits(got[1], want[1])
    assert same_bits(whole[:, 8:], before[:, 8:])  # V is as it was
    # the gradient's rotation takes it back, to the roundings of both
    back = cores.rope_backward(q, k, f, pairing=pairing)
    half = torch.finfo(DT[dt]).eps / 2
    assert bool(((back[0] - before[:, :6]).abs() <= 3 * (half + UNITS * 2.0 ** -24) * (before.abs().max() * 2)).all())


def test_only_one_in_place(cuda_ok):
    q, k = qk(64, 4, 2, 128, torch.bfloat16)
    f = cores.rope_frequencies(32)
    want = cores.rope(q, k, f)
    q2 = q.clone()
    qo, ko = cores.rope(q2, k, f, q_out=q2)
    assert same_bits(qo, want[0]) and same_bits(ko, want[1])


@pytest.mark.parametrize("pairing", ["interleaved", "half"])
def test_infinities_and_nan_stay_in_their_pairs(cuda_ok, pairing):
    q, k = qk(3, 2, 1, 64, torch.bfloat16)
    f = cores.rope_frequencies(20)
    clean = cores.rope(q, k, f, pairing=pairing)[0]
    q[1, 0, 19], q[1, 1, 30], q[2, 0, 20] = float("inf"), float("nan"), float("-inf")
    got = cores.rope(q, k, f, pairing=pairing)[0]
    mask = torch.zeros(3, 2, 64, dtype=torch.bool)
    mask[1, 0, [9, 19] if pairing == "half" else [18, 19]] = True
    mask[1, 1, 30] = mask[2, 0, 20] = True
    assert same_bits(got[~mask], clean[~mask])
    assert not torch.isfinite(got[mask]).any() and torch.isneginf(got[2, 0, 20])


def test_gradient_is_the_transpose(cuda_ok):
    # <rope(x), u> = <x, rope_backward(u)> and differences of the formula, in FP32
    x, _ = qk(20, 3, 1, 64, torch.float32)
    u, _ = qk(20, 3, 1, 64, torch.float32, seed=9)
    f = cores.rope_frequencies(48)
    for pairing in ("interleaved", "half"):
        y = f64(cores.rope(x, None, f, pairing=pairing, attention_scale=0.75)[0])
        dx = f64(cores.rope_backward(u, None, f, pairing=pairing, attention_scale=0.75)[0])
        terms = np.abs(y * f64(u)).sum() + np.abs(f64(x) * dx).sum()
        assert abs((y * f64(u)).sum() - (f64(x) * dx).sum()) <= 2 * UNITS * 2.0 ** -24 * terms
        for at in ((0, 0, 0), (7, 1, 25), (19, 2, 63)):
            e = np.zeros(x.shape)
            e[at] = 0.5  # the map is linear: any step gives the derivative
            p = steps.rope_positions(20, 20)
            d = (steps.rope(f64(x) + e, p, f64(f), pairing, 0.75)[0] - steps.rope(f64(x) - e, p, f64(f), pairing, 0.75)[0])
            assert abs((d * f64(u)).sum() - dx[at]) <= 4 * UNITS * 2.0 ** -24 * 8


@pytest.mark.parametrize("rd", [2, 20, 64, 128, 256])
def test_frequencies(cuda_ok, rd):
    for scaling, kw in (("none", {}), ("linear", {"factor": 4.0}), ("base", {"factor": 8.0}),
                        ("bands", {"factor": 8.0, "low": 1.0, "high": 4.0, "original_context": 8192.0}),
                        ("ramp", {"factor": 16.0, "low": 1.0, "high": 32.0, "original_context": 4096.0})):
        got = cores.rope_frequencies(rd, 5e5, scaling, **kw)
        want = steps.rope_frequencies(rd, 5e5, scaling, **kw)
        # the exponent's power: an error of 2^-53 of an exponent of at most 13, some 30 units of 2^-53
        assert np.all(np.abs(f64(got) - want) <= 64 * 2.0 ** -53 * want), scaling
    out = torch.zeros(rd // 2, dtype=torch.float64, device="cuda")
    assert cores.rope_frequencies(rd, 100.0, out=out) is out and float(out[0]) == 1.0


def test_decode_rows_are_the_prefill_rows(cuda_ok):
    # a token alone (its heads split over warps) and among thousands (one warp each): the same bits
    q, k = qk(6000, 8, 2, 128, torch.bfloat16)
    f = cores.rope_frequencies(128)
    for pairing in ("interleaved", "half"):
        qo, ko = cores.rope(q, k, f, pairing=pairing)
        for t in (0, 1, 4097, 5999):
            pos = torch.tensor([t], dtype=torch.int32, device="cuda")
            a, b = cores.rope(q[t:t + 1], k[t:t + 1], f, positions=pos, pairing=pairing)
            assert same_bits(a[0], qo[t]) and same_bits(b[0], ko[t])


def test_no_tokens_another_stream_and_a_graph(cuda_ok):
    f = cores.rope_frequencies(64)
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert cores.rope(none, none, f)[0].shape == (0, 2, 64)
    assert cores.rope(none.view(0, 5, 2, 64), None, f)[0].shape == (0, 5, 2, 64)
    assert cores.rope(none.view(5, 0, 2, 64), None, f)[0].shape == (5, 0, 2, 64)
    q, k = qk(100, 4, 2, 64, torch.bfloat16)
    want = cores.rope(q, k, f, pairing="half")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = cores.rope(q, k, f, pairing="half", stream=side)
    side.synchronize()
    assert same_bits(got[0], want[0]) and same_bits(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = cores.rope(q, k, f, pairing="half")
    q.copy_(-q)
    graph.replay()
    torch.cuda.synchronize()
    assert same_bits(held[0], -want[0]) and same_bits(held[1], want[1])


def test_refusals(cuda_ok):
    q, k = qk(10, 4, 2, 64, torch.bfloat16)
    f = cores.rope_frequencies(64)
    pos = torch.arange(10, dtype=torch.int32, device="cuda")
    for bad in (lambda: cores.rope(q, k, f, pairing="pairs"), lambda: cores.rope(q, k[:5], f), lambda: cores.rope(q, k.float(), f),
                lambda: cores.rope(q, k, f, positions=pos.long()), lambda: cores.rope(q, k, f, positions=pos[:9]),
                lambda: cores.rope(q, k, f.cpu()), lambda: cores.rope(q, None, f, k_out=k), lambda: cores.rope(q[0], k[0], f),
                lambda: cores.rope(q.transpose(0, 1), None, f), lambda: cores.rope(q, k, f, q_out=q[:5]),
                lambda: cores.rope(q.view(2, 5, 4, 64), None, f, cu_seqlens=pos), lambda: cores.rope_frequencies(7),
                lambda: cores.rope_frequencies(8, scaling="none", out=f), lambda: cores.rope_frequencies(8, scaling="other")):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cores.rope(q, k, f.float()), lambda: cores.rope(q.half(), None, f)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(_lib.MuseError) as e:  # a table for wider heads
        cores.rope(q, k, cores.rope_frequencies(128))
    assert e.value.status == _lib.MUSE_ERR_INVALID_ARGUMENT
