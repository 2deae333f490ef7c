"""Offsets beyond 32 bits: tensors of more than 2^31 elements, and the rows at their ends."""
import numpy as np
import pytest
import torch

from gate_cores_b200 import cores
from oracle import steps

from .close64 import f64, near, same_bits
from .test_gpu_layer_norm import BWD, FWD
from .test_gpu_rope import check

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def memory(cuda_ok):
    yield
    torch.cuda.empty_cache()


def normal(*shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(len(shape)), device="cuda", dtype=BF16)


def test_layer_norm():
    x = normal(70001, 32768)
    y = cores.layer_norm(x)
    eps = float(np.float32(1e-6))
    for part in (slice(0, 3), slice(65534, 65538), slice(69998, 70001)):  # 65536 rows: 2^31 elements, 2^32 bytes
        near(y[part], steps.layer_norm(f64(x[part]), eps=eps), FWD)
    del y
    x = x.view(-1)[:270001 * 8192].view(270001, 8192)
    dx, _, dbias = cores.layer_norm_backward(x, x)
    for part in (slice(0, 3), slice(262142, 262146), slice(269998, 270001)):
        near(dx[part], steps.layer_norm_bwd(f64(x[part]), f64(x[part]), eps=eps)[0], BWD)
    assert torch.isfinite(dbias).all()


def test_strided_rows():
    whole = torch.zeros(3 * 2 ** 31 // 2 + 4096, dtype=BF16, device="cuda")
    x = whole.as_strided((4, 1024), (2 ** 30 - 1024, 1))  # the last row begins at 3 * 2^30 elements, 2^32 bytes and more
    x.copy_(normal(4, 1024))
    want = cores.layer_norm(x.contiguous())
    assert same_bits(cores.layer_norm(x), want)
    cores.layer_norm(x, out=x)
    assert same_bits(x.contiguous(), want)
    q = x.unflatten(1, (16, 64))
    f = cores.rope_frequencies(64)
    assert same_bits(cores.rope(q, None, f)[0], cores.rope(q.contiguous(), None, f)[0])
    rows = torch.arange(4, dtype=torch.int32, device="cuda").flip(0)[:, None].contiguous()
    assert same_bits(cores.expert_combine(x, rows), x.contiguous().flip(0))
    assert same_bits(cores.expert_dispatch(x, rows), x.contiguous().flip(0))


def test_rope():
    tokens = 2 ** 31 // (16 * 128) + 333
    q = normal(tokens, 16, 128)
    f = cores.rope_frequencies(128)
    got = cores.rope(q, None, f, pairing="half")[0]
    for at in (0, 2 ** 20 - 2, tokens - 4):
        check(q[at:at + 4], got[at:at + 4], np.arange(at, at + 4), f, "half")


def test_expert_rows():
    tokens, top_k, hidden = 2 ** 18 + 77, 2, 4096 + 8
    ids = torch.randint(0, 31, (tokens, top_k), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    off, row, slot = cores.expert_sort(ids, 31)
    x = normal(tokens, hidden)
    rows = cores.expert_dispatch(x, row)
    assert rows.numel() > 2 ** 31
    for part in (slice(0, 2000), slice(-2000, None)):
        assert same_bits(rows[part], x[slot[part].long() // top_k])
    w = torch.ones(tokens, top_k, device="cuda") * 0.5
    assert same_bits(cores.expert_combine(rows, row, w), x)  # both rows of a token are its own: halves add up exactly
    dx = cores.expert_dispatch_backward(rows, row)
    assert same_bits(dx, x * 2)
    drows, dw = cores.expert_combine_backward(rows, x, row, w, drows=rows)
    for part in (slice(0, 2000), slice(-2000, None)):
        assert same_bits(drows[part], x[slot[part].long() // top_k] * 0.5)
    last = (f64(x[-9:]) ** 2).sum(-1)[:, None].repeat(top_k, 1)
    near(dw[-9:], (last, last), 48)
