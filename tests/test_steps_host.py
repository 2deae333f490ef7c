"""Host-side refusals of layer norm, rotary positions and the expert permutation, no GPU needed: every call below fails
validation (or has nothing to do) before anything is launched; its pointers are never dereferenced."""
import pytest

from gate_cores_b200 import _lib, build

INV, UNS = _lib.MUSE_ERR_INVALID_ARGUMENT, _lib.MUSE_ERR_UNSUPPORTED
BF16, F32 = _lib.MUSE_DTYPE_BF16, _lib.MUSE_DTYPE_F32
A = 0x7F0000000000  # a 256-byte aligned fake device address (never touched)
M = 1 << 24


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_layer_norm(lib):
    def ln(x=A, y=A + M, dt=BF16, rows=4, hidden=256, xs=None, ys=None, gain=A + 2 * M, off=0.0, bias=A + 3 * M, eps=1e-6):
        return lib.muse_layer_norm(x, y, dt, rows, hidden, hidden if xs is None else xs, hidden if ys is None else ys,
                                   gain, off, bias, eps, None)

    assert ln(rows=0) == 0 and ln(rows=0, x=None, y=None) == 0
    assert ln(dt=7) == INV and ln(rows=-1) == INV and ln(hidden=0) == INV
    assert ln(x=None) == INV and ln(y=None) == INV
    assert ln(xs=248) == INV and ln(ys=248) == INV
    assert ln(eps=-1e-6) == INV and ln(eps=float("nan")) == INV and ln(off=float("inf")) == INV
    assert ln(x=A + 8) == UNS and ln(hidden=252) == UNS and ln(xs=260) == UNS and ln(hidden=32776) == UNS
    assert ln(gain=A + 2 * M + 8) == UNS and ln(bias=A + 3 * M + 4) == UNS
    assert ln(y=A + 256) == INV                       # partly over x
    assert ln(y=A + 2 * M) == INV and ln(y=A + 3 * M) == INV  # over the gain, over the bias
    assert b"muse_layer_norm" in lib.muse_last_error()


def test_layer_norm_backward(lib):
    need = lib.muse_norm_backward_workspace_bytes(64, 256)

    def bwd(x=A, dy=A + M, dx=A + 2 * M, dt=BF16, rows=64, hidden=256, xs=256, gain=A + 3 * M, eps=1e-6, dgain=A + 4 * M,
            dbias=A + 5 * M, ws=A + 6 * M, n=need):
        return lib.muse_layer_norm_backward(x, dy, dx, dt, rows, hidden, xs, hidden, hidden, gain, 0.0, eps, dgain, dbias,
                                            ws, n, None)

    assert bwd(rows=0, dgain=None, dbias=None) == 0
    assert bwd(gain=None) == INV                      # a gain's gradient without a gain
    assert bwd(ws=None) == INV and bwd(n=need - 1) == INV and bwd(dgain=None, n=need - 1) == INV
    assert bwd(ws=A + 6 * M + 8) == UNS and bwd(dbias=A + 5 * M + 8) == UNS and bwd(dgain=A + 4 * M + 4) == UNS
    assert bwd(xs=248) == INV and bwd(dx=None) == INV and bwd(eps=float("inf")) == INV
    assert bwd(hidden=8200, xs=8200) == UNS           # above 1024 vectors
    assert bwd(dx=A + 512) == INV and bwd(dx=A + 3 * M) == INV
    assert bwd(dbias=A + 4 * M) == INV                # both gradients in one place
    assert bwd(dbias=A) == INV and bwd(dbias=A + 6 * M) == INV and bwd(dgain=A + M) == INV
    assert bwd(ws=A + M) == INV
