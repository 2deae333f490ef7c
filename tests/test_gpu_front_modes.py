"""PyTorch's modes see the outputs of the calls as they see other new tensors."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from gate_cores_b200 import cores

from .close64 import same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture
def deterministic():
    was, fill = torch.are_deterministic_algorithms_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    torch.use_deterministic_algorithms(True)
    torch.utils.deterministic.fill_uninitialized_memory = True
    yield
    torch.use_deterministic_algorithms(was)
    torch.utils.deterministic.fill_uninitialized_memory = fill


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rows_that_nothing_writes_are_filled(cuda_ok, deterministic, dt):
    x = torch.ones(5, 64, dtype=dt, device="cuda")
    row = torch.tensor([[0, 1], [-1, 2], [-1, -1], [3, -1], [4, -1]], dtype=torch.int32, device="cuda")
    # (memory that comes back from the allocator with something in it)
    for _ in range(3):
        torch.full((10, 64), 7.0, dtype=dt, device="cuda")
        rows = cores.expert_dispatch(x, row)
        drows, dw = cores.expert_combine_backward(torch.ones_like(rows), x, row)
        for t in (rows, drows):
            assert bool((t[:5] == 1).all()) and bool(torch.isnan(t[5:]).all())


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.shapes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func._schema.name.startswith("aten::empty"):
            self.shapes.append(tuple(out.shape))
        return out


def test_a_dispatch_mode_sees_the_outputs(cuda_ok):
    x = torch.randn(300, 64, device="cuda")
    ids = torch.zeros(300, 2, dtype=torch.int32, device="cuda")
    f = cores.rope_frequencies(64)
    want = cores.layer_norm(x), *cores.layer_norm_backward(x, x, x[0].contiguous()), *cores.expert_sort(ids, 4)
    with Seen() as seen:
        got = cores.layer_norm(x), *cores.layer_norm_backward(x, x, x[0].contiguous()), *cores.expert_sort(ids, 4)
        row = got[5]
        rows = cores.expert_dispatch(x, row)
        y = cores.expert_combine(rows, row)
        drows, dw = cores.expert_combine_backward(rows, y, row)
        q, _ = cores.rope(x.view(300, 1, 64), None, f)
    assert all(same_bits(a, b) for a, b in zip(want, got))
    assert len(seen.shapes) >= 12  # an output each, workspaces beside them
    for t in (*got, rows, y, drows, dw, q):
        assert tuple(t.shape) in seen.shapes
