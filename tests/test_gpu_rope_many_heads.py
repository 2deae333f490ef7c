"""Rotary positions where a warp takes more of a token's heads than it has loads on their way: places refilled, heads
brought to shared memory in several rounds.  Tolerances as in test_gpu_rope.py."""
import pytest
import torch

from gate_cores_b200 import cores
from oracle import steps

from .close64 import same_bits
from .test_gpu_rope import DT, check, qk

pytestmark = pytest.mark.gpu

TOKENS = 2500  # a warp each, on 148 SMs (fewer tokens are shared by several)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hq,hk,d,rd,pairing", [
    (40, 8, 128, 64, "interleaved"), (40, 8, 128, 128, "interleaved"), (40, 8, 128, 128, "half"), (40, 8, 128, 64, "half"),
    (32, 8, 80, 20, "half"), (41, 3, 80, 36, "half"), (37, 0, 64, 4, "half"), (33, 7, 96, 20, "interleaved"), (64, 64, 64, 64, "half"),
    (1, 70, 128, 128, "half")])
@pytest.mark.parametrize("backward", [False, True], ids=["fwd", "bwd"])
def test_many_heads(cuda_ok, dt, hq, hk, d, rd, pairing, backward):
    q, k = qk(TOKENS, hq, max(hk, 1), d, DT[dt], fused=True)
    k = k if hk else None
    whole = q._base if q._base is not None else q
    before = whole.clone()
    f = cores.rope_frequencies(rd, 1e4)
    pos = (torch.arange(TOKENS, dtype=torch.int32) * 977 % 131072).cuda()
    call = cores.rope_backward if backward else cores.rope
    got = call(q, k, f, positions=pos, pairing=pairing)
    host = pos.cpu().numpy()
    for x, y in zip((q, k), got):
        if x is not None:
            check(x, y, host, f, pairing, 1.0, backward)
            assert same_bits(y[..., rd:], x[..., rd:])
    assert same_bits(whole, before)
    # in place on the projection, what is behind Q and K as it was
    again = call(q, k, f, pos, None, pairing, 1.0, q, k)
    assert same_bits(again[0], got[0]) and (k is None or same_bits(again[1], got[1]))
    assert same_bits(whole[:, hq + hk:], before[:, hq + hk:])


@pytest.mark.parametrize("pairing,rd", [("interleaved", 64), ("half", 128), ("half", 20)])
def test_many_heads_of_packed_documents(cuda_ok, pairing, rd):
    lengths = [1, 999, 0, 700, 800]
    cu = torch.tensor([0] + lengths).cumsum(0).to(torch.int32)
    q, k = qk(TOKENS, 24, 24, 128, torch.bfloat16)
    f = cores.rope_frequencies(rd, 5e5)
    got = cores.rope(q, k, f, cu_seqlens=cu.cuda(), pairing=pairing)
    pos = steps.rope_positions(TOKENS, cu_seqlens=cu.numpy())
    check(q, got[0], pos, f, pairing)
    check(k, got[1], pos, f, pairing)
