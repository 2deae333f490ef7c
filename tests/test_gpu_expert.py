"""Tokens sorted by expert and back, on the GPU, against the float64 formulas.

Units of 2^-24 (tests/close64.py): combine: a product and a sum for each of top_k terms, of the sum of their magnitudes:
2 top_k <= 32; dispatch's backward the sums alone.  drows: one product, which for FP32 is the output's own rounding and
for bf16 one unit before it: 1.  dweights: a sum of H <= 8192 products, at most 32 in a row in a thread (and as many
joins of chains), 5 + 3 in the butterflies: 48 with the products.
"""
import numpy as np
import pytest
import torch

from gate_cores_b200 import _lib, cores
from oracle import steps

from .close64 import f64, near, same_bits

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def choices(tokens, top_k, experts, seed=0, dropped=0.0, dtype=torch.int32, skew=2.0):
    g = torch.Generator().manual_seed(seed + tokens * 7 + experts)
    score = torch.rand(tokens, experts, generator=g) ** (0.2 + skew * torch.rand(experts, generator=g))
    ids = score.topk(top_k, dim=1).indices if top_k <= experts else torch.randint(0, experts, (tokens, top_k), generator=g)
    if dropped:
        ids = torch.where(torch.rand(tokens, top_k, generator=g) < dropped, torch.randint(-3, 0, (tokens, top_k), generator=g), ids)
    return ids.to(dtype)


def values(rows, hidden, dt, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 31 + hidden)
    return torch.randn(rows, hidden, generator=g).to(dt).cuda()


def check_sort(ids, experts, got):
    off, row, slot = steps.expert_sort(ids.cpu().numpy(), experts)
    assert np.array_equal(got[0].cpu().numpy(), off)
    assert np.array_equal(got[1].cpu().numpy(), row)
    assert np.array_equal(got[2].cpu().numpy(), slot)


# one slot, less than a warp, odd sizes, one CTA of either kind exactly and one slot more, many CTAs of either, many experts
SORTS = [(1, 1, 1), (3, 2, 4), (37, 3, 5), (128, 8, 64), (1025, 1, 9), (1024, 4, 33), (4097, 1, 7), (151552, 1, 64), (151553, 1, 64), (1366, 3, 1024), (20000, 8, 64), (9001, 5, 300)]


@pytest.mark.parametrize("tokens,top_k,experts", SORTS)
@pytest.mark.parametrize("dropped", [0.0, 0.3])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(cuda_ok, tokens, top_k, experts, dropped, dtype):
    ids = choices(tokens, top_k, experts, dropped=dropped, dtype=dtype)
    check_sort(ids, experts, cores.expert_sort(ids.cuda(), experts))


def test_sort_odd_choices(cuda_ok):
    for ids, experts in ((torch.full((300, 4), 2), 5), (torch.full((300, 4), -1), 5), (torch.full((3000, 4), 7), 7),
                         (torch.tensor([[2 ** 32 + 1, 1], [1, -2 ** 40]]), 3), (torch.tensor([[0, 0, 0], [1, 0, 1]]), 2),
                         (torch.arange(5000)[:, None] % 1024, 1024), (4999 - torch.arange(5000)[:, None], 1000)):
        check_sort(ids, experts, cores.expert_sort(ids.cuda(), experts))
    none = cores.expert_sort(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 9)
    assert none[0].shape == (10,) and not none[0].any() and none[1].shape == (0, 4) and none[2].shape == (0,)
    wide = choices(100, 6, 8).cuda()
    check_sort(wide[:, 1:4], 8, cores.expert_sort(wide[:, 1:4], 8))  # not contiguous


def test_sort_is_large(cuda_ok):
    # more than 512 CTAs' worth of slots (longer runs a CTA), against a stable sort
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(-1, 97, (700001, 4), generator=g, device="cuda", dtype=torch.int32)
    off, row, slot = cores.expert_sort(ids, 97)
    flat = torch.where(ids.reshape(-1) < 0, 97, ids.reshape(-1))
    order = torch.sort(flat, stable=True).indices
    kept = int((flat < 97).sum())
    assert torch.equal(slot[:kept].long(), order[:kept]) and bool((slot[kept:] == -1).all())
    assert torch.equal(off.long(), torch.searchsorted(flat[order], torch.arange(98, device="cuda")))
    assert torch.equal(row.reshape(-1)[order[:kept]].long(), torch.arange(kept, device="cuda"))
    assert bool((row[ids < 0] == -1).all())


# odd tokens, one vector, odd vectors, rows of one CTA's width and more
ROWS = [(1, 1, 1, 8), (7, 2, 3, 40), (37, 3, 5, 264), (128, 8, 64, 4096), (501, 4, 16, 1000), (65, 6, 9, 5120), (33, 9, 12, 2056),
        (19, 16, 16, 8192)]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("tokens,top_k,experts,hidden", ROWS)
@pytest.mark.parametrize("dropped", [0.0, 0.4])
def test_rows_there_and_back(cuda_ok, dt, tokens, top_k, experts, hidden, dropped):
    ids = choices(tokens, top_k, experts, dropped=dropped).cuda()
    off, row, slot = cores.expert_sort(ids, experts)
    kept, n = int(off[-1]), tokens * top_k
    x, made, dy = values(tokens, hidden, DT[dt]), values(n, hidden, DT[dt], 1), values(tokens, hidden, DT[dt], 2)
    w = torch.softmax(values(tokens, top_k, torch.float32, 3), 1)
    host = row.cpu().numpy()

    into = torch.full((n, hidden), 9.0, dtype=DT[dt], device="cuda")
    assert cores.expert_dispatch(x, row, out=into) is into
    assert same_bits(into[:kept], x[slot[:kept].long() // top_k]) and bool((into[kept:] == 9.0).all())
    assert same_bits(cores.expert_dispatch(x, row)[:kept], into[:kept])

    made[kept:] = float("nan")  # behind the last group: not read
    near(cores.expert_combine(made, row, w), steps.expert_combine(f64(made), host, f64(w)), 32, "combine")
    near(cores.expert_combine(made, row), steps.expert_combine(f64(made), host), 32, "combine, no weights")
    near(cores.expert_dispatch_backward(made, row), steps.expert_combine(f64(made), host), 32, "dispatch backward")

    for weights in (w, None):
        (rd, rdm), rw = steps.expert_combine_bwd(f64(made), f64(dy), host, None if weights is None else f64(weights))
        drows = torch.full((n, hidden), 5.0, dtype=DT[dt], device="cuda")
        got, dw = cores.expert_combine_backward(made, dy, row, weights, drows=drows)
        assert got is drows and bool((got[kept:] == 5.0).all())
        near(got[:kept], (rd[:kept], rdm[:kept]), 1, "drows")
        near(dw, rw, 48, "dweights")
        assert not dw[row < 0].any()
        only, none = cores.expert_combine_backward(made, dy, row, weights, want_dweights=False)
        assert none is None and same_bits(only[:kept], got[:kept])
    # in place over the rows
    copy = made.clone()
    again, dw2 = cores.expert_combine_backward(copy, dy, row, None, drows=copy)
    assert same_bits(again[:kept], got[:kept]) and same_bits(dw2, dw)


def test_tokens_without_rows_and_rows_out_of_range(cuda_ok):
    row = torch.tensor([[0, 1], [-1, -1], [2, 99], [3, -7], [2 ** 31 - 1, 4]], dtype=torch.int32, device="cuda")
    made, dy = values(5, 64, torch.bfloat16), values(5, 64, torch.bfloat16, 1)
    w = torch.full((5, 2), 0.5, device="cuda")
    w[1] = float("inf")  # a dropped slot's weight does not matter
    y = cores.expert_combine(made, row, w)
    near(y, steps.expert_combine(f64(made), row.cpu().numpy(), np.full((5, 2), 0.5)), 4)
    assert not y[1].any()
    drows, dw = cores.expert_combine_backward(made, dy, row, w)
    assert not dw[1].any() and dw[2, 1] == 0 and dw[4, 0] == 0 and bool(torch.isfinite(drows).all())
    # fewer rows than slots: the slots beyond them are dropped
    few = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    cores.expert_dispatch(dy, row, out=few)
    assert same_bits(few, dy[[0, 0]])
    assert not cores.expert_combine(made[:0], row).any()


def test_infinite_rows_stay_with_their_tokens(cuda_ok):
    ids = choices(50, 2, 4).cuda()
    _, row, _ = cores.expert_sort(ids, 4)
    made = values(100, 128, torch.bfloat16)
    clean = cores.expert_combine(made, row)
    r = int(row[10, 1])
    made[r, 5] = float("inf")
    y = cores.expert_combine(made, row)
    assert torch.isinf(y[10, 5])
    y[10, 5] = clean[10, 5]
    assert same_bits(y, clean)


@pytest.mark.parametrize("dt", DT)
def test_strides(cuda_ok, dt):
    ids = choices(60, 3, 6).cuda()
    _, row, _ = cores.expert_sort(ids, 6)
    wide, rows = values(60, 512, DT[dt]), values(180, 768, DT[dt], 1)
    x, made = wide[:, 128:384], rows[:, 256:512]
    w = torch.rand(60, 6, device="cuda")[:, ::2]
    out = torch.full((180, 512), 2.0, dtype=DT[dt], device="cuda")
    cores.expert_dispatch(x, row, out=out[:, :256])
    assert same_bits(out[:, :256], cores.expert_dispatch(x.contiguous(), row)) and bool((out[:, 256:] == 2.0).all())
    y = torch.full((60, 512), 2.0, dtype=DT[dt], device="cuda")
    cores.expert_combine(made, row, w, out=y[:, 256:])
    assert same_bits(y[:, 256:], cores.expert_combine(made.contiguous(), row, w.contiguous())) and bool((y[:, :256] == 2.0).all())
    a = cores.expert_combine_backward(made, x, row, w)
    b = cores.expert_combine_backward(made.contiguous(), x.contiguous(), row, w.contiguous())
    assert same_bits(a[0], b[0]) and same_bits(a[1], b[1])


def test_gradients_against_differences(cuda_ok):
    # loss = <combine(rows, w), u>, with rows and w moved; loss = <dispatch(x), v>, with x moved (all linear: any step)
    ids = choices(9, 2, 3, dropped=0.2).cuda()
    off, row, _ = cores.expert_sort(ids, 3)
    host, kept = row.cpu().numpy(), int(off[-1])
    made, u, w = values(18, 16, torch.float32), values(9, 16, torch.float32, 1), torch.rand(9, 2).cuda()
    drows, dw = cores.expert_combine_backward(made, u, row, w)
    for r, h in ((0, 0), (kept - 1, 15), (kept // 2, 7)):
        e = np.zeros((18, 16))
        e[r, h] = 0.5
        d = steps.expert_combine(f64(made) + e, host, f64(w))[0] - steps.expert_combine(f64(made) - e, host, f64(w))[0]
        assert abs((d * f64(u)).sum() - float(drows[r, h])) <= 4 * 2.0 ** -24 * 8
    for t, j in ((0, 0), (5, 1), (8, 0)):
        e = np.zeros((9, 2))
        e[t, j] = 0.5
        d = steps.expert_combine(f64(made), host, f64(w) + e)[0] - steps.expert_combine(f64(made), host, f64(w) - e)[0]
        assert abs((d * f64(u)).sum() - float(dw[t, j])) <= 48 * 2.0 ** -24 * 64
    v = values(18, 16, torch.float32, 4)
    dx = cores.expert_dispatch_backward(v, row)
    x = values(9, 16, torch.float32, 5)
    for t, h in ((0, 3), (4, 0), (8, 15)):
        moved = x.clone()
        moved[t, h] += 1.0
        d = f64(cores.expert_dispatch(moved, row)[:kept]) - f64(cores.expert_dispatch(x, row)[:kept])
        # x + 1 is rounded once, its difference from x is then exact to that
        assert abs((d * f64(v)[:kept]).sum() - float(dx[t, h])) <= 8 * 2.0 ** -24 * 16


def test_another_stream_and_graphs(cuda_ok):
    ids = choices(3000, 4, 32).cuda()  # several CTAs: the sort has a workspace
    x = values(3000, 256, torch.bfloat16)
    w = torch.rand(3000, 4, device="cuda")

    def all_of(stream=None):
        off, row, slot = cores.expert_sort(ids, 32, stream=stream)
        rows = cores.expert_dispatch(x, row, stream=stream)
        y = cores.expert_combine(rows, row, w, stream=stream)
        return (off, row, slot, rows, y, *cores.expert_combine_backward(rows, y, row, w, stream=stream),
                cores.expert_dispatch_backward(rows, row, stream=stream))

    want = all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = all_of(side)
    side.synchronize()
    assert all(same_bits(a, b) for a, b in zip(want, got))
    # two captured graphs that share one workspace, replayed in turn
    ws = torch.empty(_lib.muse_expert_sort_workspace_bytes(12000, 32), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    other = choices(3000, 4, 32, seed=5).cuda()
    graphs, held = [], []
    for i in (ids, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(cores.expert_sort(i, 32, workspace=ws))
        graphs.append(g)
    for k in (0, 1, 0):
        graphs[k].replay()
    torch.cuda.synchronize()
    for i, h in zip((ids, other), held):
        check_sort(i, 32, h)


def test_refusals(cuda_ok):
    ids = choices(10, 2, 4).cuda()
    _, row, _ = cores.expert_sort(ids, 4)
    x, rows = values(10, 64, torch.bfloat16), values(20, 64, torch.bfloat16)
    w = torch.rand(10, 2, device="cuda")
    for bad in (lambda: cores.expert_sort(ids[0], 4), lambda: cores.expert_sort(ids, 0), lambda: cores.expert_sort(ids.cpu(), 4),
                lambda: cores.expert_dispatch(x[:9], row), lambda: cores.expert_dispatch(x, row.long()),
                lambda: cores.expert_dispatch(x, row, out=rows[:, :32]), lambda: cores.expert_dispatch(x, row, out=rows.float()),
                lambda: cores.expert_combine(rows, row, w[:9]), lambda: cores.expert_combine(rows, row, out=x[:9]),
                lambda: cores.expert_combine(rows[None], row), lambda: cores.expert_combine_backward(rows, x.float(), row),
                lambda: cores.expert_combine_backward(rows, x[:, :32], row),
                lambda: cores.expert_combine_backward(rows, x, row, drows=rows[:19])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cores.expert_sort(ids.float(), 4), lambda: cores.expert_combine(rows, row, w.double()),
                lambda: cores.expert_dispatch(x.half(), row)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(_lib.MuseError) as e:
        cores.expert_sort(ids, 1025)
    assert e.value.status == _lib.MUSE_ERR_UNSUPPORTED
    with pytest.raises(_lib.MuseError) as e:
        cores.expert_combine(rows, row, out=rows[:10])
    assert e.value.status == _lib.MUSE_ERR_INVALID_ARGUMENT


def test_a_workspace_that_is_not_its_own_bytes(cuda_ok):
    ids = choices(12000, 1, 32).cuda()
    need = _lib.muse_expert_sort_workspace_bytes(12000, 32)
    whole = torch.empty(2 * need, dtype=torch.uint8, device="cuda")
    for ws in (whole[:1].expand(need), whole[::2], whole[:need - 1]):
        with pytest.raises(ValueError):
            cores.expert_sort(ids, 32, workspace=ws)


def test_choices_written_just_before(cuda_ok):
    # one buffer, other choices before each sort, nothing waited for
    many = [choices(6000, 4, 64, seed=s).cuda() for s in range(24)]
    ids = torch.empty_like(many[0])
    ws = torch.empty(_lib.muse_expert_sort_workspace_bytes(24000, 64), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = []
    for i in many:
        ids.copy_(i)
        got.append(cores.expert_sort(ids, 64, workspace=ws))
    torch.cuda.synchronize()
    for i, g in zip(many, got):
        check_sort(i, 64, g)


# around the sizes where the steps of a CTA and the way to its first rows change
@pytest.mark.parametrize("slots,experts", [(303104, 17), (303104, 18), (303105, 100), (303105, 110), (757760, 1), (757761, 64),
                                           (40000, 1000), (39000, 1024), (2097153, 3), (2500001, 64)])
def test_sort_where_its_shape_changes(cuda_ok, slots, experts):
    ids = choices(slots, 1, experts, seed=slots + experts).cuda()
    check_sort(ids, experts, cores.expert_sort(ids, experts))
