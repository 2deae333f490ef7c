"""What is not rotated leaves with the bits it came with, NaN and their payloads too, also where it shares 16 bytes with
what is."""
import pytest
import torch

from gate_cores_b200 import cores

from .close64 import same_bits

pytestmark = pytest.mark.gpu

# every kind of 16-bit and 32-bit pattern that a conversion might change: NaN quiet and not, of both signs, infinities,
# zeros of both signs, the smallest numbers
PATTERNS = {torch.bfloat16: [0x7FA5, 0xFF81, 0x7FC1, 0xFFFF, 0x7F80, 0xFF80, 0x8000, 0x0001, 0x8001, 0x3F80],
            torch.float32: [0x7FA00005, 0xFF800001, 0x7FC00001, 0xFFFFFFFF, 0x7F800000, 0xFF800000, 0x80000000, 0x00000001,
                            0x80000001, 0x3F800000]}


@pytest.mark.parametrize("dt", list(PATTERNS), ids=["bf16", "f32"])
@pytest.mark.parametrize("pairing,d,rd", [("interleaved", 64, 20), ("interleaved", 64, 18), ("interleaved", 64, 22), ("interleaved", 64, 2),
                                          ("interleaved", 64, 16), ("half", 64, 20), ("half", 64, 16), ("half", 80, 36)])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("backward", [False, True], ids=["fwd", "bwd"])
def test_bits_behind_the_rotated_part(cuda_ok, dt, pairing, d, rd, in_place, backward):
    ints = torch.int16 if dt == torch.bfloat16 else torch.int32
    wide = torch.tensor(PATTERNS[dt], dtype=torch.int64)
    top = 1 << (16 if dt == torch.bfloat16 else 32)
    wide = torch.where(wide >= top // 2, wide - top, wide).to(ints)
    g = torch.Generator().manual_seed(d + rd)
    q = torch.randn(23, 5, d, generator=g).to(dt)
    k = torch.randn(23, 2, d, generator=g).to(dt)
    for t in (q, k):
        n = t[..., rd:].numel()
        t.view(ints)[..., rd:] = wide[torch.randint(0, len(wide), (n,), generator=g)].view(t[..., rd:].shape)
    q, k = q.cuda(), k.cuda()
    behind = q[..., rd:].clone(), k[..., rd:].clone()
    call = cores.rope_backward if backward else cores.rope
    got = call(q, k, cores.rope_frequencies(rd), None, None, pairing, 1.0, *((q, k) if in_place else (None, None)))
    for y, b in zip(got, behind):
        assert same_bits(y[..., rd:], b)
        assert torch.isfinite(y[..., :rd].float()).all()
