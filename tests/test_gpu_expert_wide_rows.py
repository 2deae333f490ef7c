"""The experts' rows where a token's threads go over its row more than once: more tokens than get threads for their whole
row, rows wider than 256 threads take at a time.  Tolerances as in test_gpu_expert.py."""
import pytest
import torch

from gate_cores_b200 import cores
from oracle import steps

from .close64 import f64, near, same_bits
from .test_gpu_expert import DT, choices, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("top_k", [1, 2, 3, 8])
@pytest.mark.parametrize("hidden", [4104, 8192])
def test_wide_rows_of_many_tokens(cuda_ok, dt, top_k, hidden):
    tokens, experts = 411, 16
    ids = choices(tokens, top_k, experts, dropped=0.1).cuda()
    off, row, slot = cores.expert_sort(ids, experts)
    kept, n = int(off[-1]), tokens * top_k
    x, made, dy = values(tokens, hidden, DT[dt]), values(n, hidden, DT[dt], 1), values(tokens, hidden, DT[dt], 2)
    w = torch.softmax(values(tokens, top_k, torch.float32, 3), 1)
    host = row.cpu().numpy()
    into = torch.full((n, hidden), 9.0, dtype=DT[dt], device="cuda")
    cores.expert_dispatch(x, row, out=into)
    assert same_bits(into[:kept], x[slot[:kept].long() // top_k]) and bool((into[kept:] == 9.0).all())
    made[kept:] = float("nan")
    made64, dy64 = f64(made), f64(dy)
    near(cores.expert_combine(made, row, w), steps.expert_combine(made64, host, f64(w)), 32, "combine")
    plain = steps.expert_combine(made64, host)
    near(cores.expert_combine(made, row), plain, 32, "combine, no weights")
    near(cores.expert_dispatch_backward(made, row), plain, 32, "dispatch backward")
    (rd, rdm), rw = steps.expert_combine_bwd(made64, dy64, host, f64(w))
    drows, dw = cores.expert_combine_backward(made, dy, row, w)
    near(drows[:kept], (rd[:kept], rdm[:kept]), 1, "drows")
    near(dw, rw, 48, "dweights")
    again, dw2 = cores.expert_combine_backward(made, dy, row, w, drows=made)  # in place
    assert same_bits(again[:kept], drows[:kept]) and same_bits(dw2, dw)
