"""Comparison of the library's outputs with a float64 reference.

A floating output is the rounding to its dtype (half a step of it: finfo.eps / 2 of the value) of an FP32 evaluation,
which is off by at most `units` * 2^-24 of `mag`, the magnitudes that the evaluation rounds.  How many units an
operator takes is counted at its tests.
"""
import numpy as np
import torch

HALF_STEP = {dt: torch.finfo(dt).eps / 2 for dt in (torch.bfloat16, torch.float32)}  # 2^-8, 2^-24


def f64(t: torch.Tensor) -> np.ndarray:
    """The exact values of a tensor."""
    return t.detach().to(torch.float64).cpu().numpy()


def near(got: torch.Tensor, ref, units: float, what: str = ""):
    want, mag = ref
    g = f64(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    off = units * 2.0 ** -24 * mag
    tol = off + HALF_STEP[got.dtype] * (np.abs(want) + off)
    # written so that a NaN fails
    bad = np.flatnonzero(~(np.abs(g - want) <= tol).ravel())
    if bad.size:
        i = bad[:6]
        raise AssertionError(f"{what}: {bad.size} of {g.size} off; at {i.tolist()} got {g.ravel()[i].tolist()} "
                             f"want {want.ravel()[i].tolist()} within {np.broadcast_to(tol, g.shape).ravel()[i].tolist()}")


def same_bits(a: torch.Tensor, b: torch.Tensor) -> bool:
    view = {2: torch.int16, 4: torch.int32, 8: torch.int64}[a.element_size()]
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(a.contiguous().view(view), b.contiguous().view(view))
