"""The calls by device address (_lib) of layer norm, the rotary positions and the experts' rows, for programs whose memory
is not PyTorch's: the same bits as the tensor calls, on a stream given by its number."""
import pytest
import torch

from gate_cores_b200 import _lib, cores

from .close64 import same_bits

pytestmark = pytest.mark.gpu

BF16, F32 = _lib.MUSE_DTYPE_BF16, _lib.MUSE_DTYPE_F32


def test_every_entry_point_has_a_call():
    for name in _lib.EXPORTS:
        assert callable(getattr(_lib, name)), name


@pytest.fixture
def stream(cuda_ok):
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    yield s.cuda_stream
    torch.cuda.synchronize()


def test_layer_norm(stream):
    x, dy = torch.randn(70, 1000, device="cuda").bfloat16(), torch.randn(70, 1000, device="cuda").bfloat16()
    g, b = torch.randn(1000, device="cuda"), torch.randn(1000, device="cuda")
    want = cores.layer_norm(x, g, b, 0.5, 1e-5), *cores.layer_norm_backward(x, dy, g, 0.5, 1e-5)
    got = tuple(torch.empty_like(t) for t in want)
    n = _lib.muse_norm_backward_workspace_bytes(70, 1000)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    _lib.muse_layer_norm(x.data_ptr(), got[0].data_ptr(), BF16, 70, 1000, 1000, 1000, g.data_ptr(), 0.5, b.data_ptr(), 1e-5, stream)
    _lib.muse_layer_norm_backward(x.data_ptr(), dy.data_ptr(), got[1].data_ptr(), BF16, 70, 1000, 1000, 1000, 1000, g.data_ptr(), 0.5,
                                  1e-5, got[2].data_ptr(), got[3].data_ptr(), ws.data_ptr(), n, stream)
    torch.cuda.synchronize()
    assert all(same_bits(a, c) for a, c in zip(want, got))


def test_rope(stream):
    q, k = torch.randn(30, 4, 64, device="cuda"), torch.randn(30, 2, 64, device="cuda")
    f, at = cores.rope_frequencies(32), torch.arange(30, device="cuda", dtype=torch.int32) * 91
    for call, raw in ((cores.rope, _lib.muse_rope), (cores.rope_backward, _lib.muse_rope_backward)):
        want = call(q, k, f, at, pairing="half", attention_scale=1.5)
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        torch.cuda.synchronize()
        raw(q.data_ptr(), k.data_ptr(), qo.data_ptr(), ko.data_ptr(), F32, _lib.MUSE_LAYOUT_BSHD, 1, 30, None, 0, 30, at.data_ptr(), 4, 2,
            64, 32, _lib.MUSE_ROPE_HALVES, 256, 128, 256, 128, f.data_ptr(), 1.5, stream)
        torch.cuda.synchronize()
        assert same_bits(qo, want[0]) and same_bits(ko, want[1])


def test_experts(stream):
    T, K, E, H = 3000, 3, 40, 136
    ids = torch.randint(-1, E, (T, K), device="cuda")
    x, w = torch.randn(T, H, device="cuda").bfloat16(), torch.rand(T, K, device="cuda")
    off, row, slot = cores.expert_sort(ids, E)
    kept = int(off[-1])
    got = torch.empty_like(off), torch.empty_like(row), torch.empty_like(slot)
    n = _lib.muse_expert_sort_workspace_bytes(T * K, E)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    rows, y, dx, dw = (torch.empty(s, dtype=d, device="cuda") for s, d in (((T * K, H), x.dtype), ((T, H), x.dtype), ((T, H), x.dtype),
                                                                            ((T, K), torch.float32)))
    drows = torch.empty_like(rows)
    torch.cuda.synchronize()
    _lib.muse_expert_sort(ids.data_ptr(), _lib.MUSE_INDEX_I64, T, K, E, *(t.data_ptr() for t in got), ws.data_ptr(), n, stream)
    r = got[1].data_ptr()
    _lib.muse_expert_dispatch(x.data_ptr(), rows.data_ptr(), BF16, T, H, K, T * K, H, H, r, stream)
    _lib.muse_expert_combine(rows.data_ptr(), y.data_ptr(), BF16, T, H, K, T * K, H, H, r, w.data_ptr(), stream)
    _lib.muse_expert_combine_backward(rows.data_ptr(), x.data_ptr(), drows.data_ptr(), BF16, T, H, K, T * K, H, H, H, r, w.data_ptr(),
                                      dw.data_ptr(), stream)
    _lib.muse_expert_dispatch_backward(drows.data_ptr(), dx.data_ptr(), BF16, T, H, K, T * K, H, H, r, stream)
    torch.cuda.synchronize()
    assert all(same_bits(a, c) for a, c in zip((off, row, slot), got))
    want = cores.expert_dispatch(x, row)
    assert same_bits(rows[:kept], want[:kept]) and same_bits(y, cores.expert_combine(want, row, w))
    wd, ww = cores.expert_combine_backward(want, x, row, w)
    assert same_bits(drows[:kept], wd[:kept]) and same_bits(dw, ww)
    assert same_bits(dx, cores.expert_dispatch_backward(wd, row))
