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


def test_rope(lib):
    def rope(q=A, k=A + M, qo=A + 2 * M, ko=A + 3 * M, dt=BF16, layout=0, batch=2, seqlen=8, cu=None, ns=0, total=16, pos=None,
             hq=4, hk=2, d=64, rd=64, pairing=1, qs=None, ks=None, qos=None, kos=None, f=A + 4 * M, scale=1.0, fn=None):
        return (fn or lib.muse_rope)(q, k, qo, ko, dt, layout, batch, seqlen, cu, ns, total, pos, hq, hk, d, rd, pairing,
                                     hq * d if qs is None else qs, hk * d if ks is None else ks, hq * d if qos is None else qos,
                                     hk * d if kos is None else kos, f, scale, None)

    assert rope(batch=0) == 0 and rope(batch=0, seqlen=0, q=None, k=None, f=None) == 0
    assert rope(layout=1, total=0) == 0
    assert rope(dt=5) == INV and rope(layout=2) == INV and rope(pairing=2) == INV and rope(pairing=-1) == INV
    assert rope(batch=-1) == INV and rope(seqlen=0) == INV and rope(layout=1, total=-1) == INV
    assert rope(hq=0) == INV and rope(hk=-1) == INV and rope(d=0, rd=0) == INV
    assert rope(rd=0) == INV and rope(rd=63) == INV and rope(rd=66) == INV
    assert rope(scale=float("nan")) == INV and rope(scale=float("inf")) == INV
    assert rope(qs=248) == INV and rope(ks=120) == INV and rope(qos=0) == INV and rope(kos=64) == INV
    assert rope(layout=1) == INV and rope(layout=1, cu=A + 5 * M) == INV
    assert rope(q=None) == INV and rope(k=None) == INV and rope(ko=None) == INV and rope(f=None) == INV
    assert rope(q=A + 8) == UNS and rope(ko=A + 3 * M + 2) == UNS and rope(d=68, rd=64) == UNS and rope(qs=260) == UNS
    assert rope(d=264, rd=64) == UNS and rope(dt=F32, d=132, rd=64) == UNS
    assert rope(f=A + 4 * M + 4) == UNS and rope(pos=A + 5 * M + 2) == UNS and rope(layout=1, cu=A + 5 * M + 1, ns=1) == UNS
    assert rope(batch=1 << 40, seqlen=1 << 40) == UNS and rope(layout=1, total=1 << 31, pos=A + (1 << 60)) == UNS
    assert rope(hq=1 << 23) == UNS
    assert rope(qo=A + 128) == INV and rope(qo=A + M) == INV and rope(ko=A) == INV and rope(ko=A + 2 * M) == INV
    assert rope(f=A + 2 * M) == INV and rope(pos=A + 3 * M) == INV and rope(layout=1, cu=A + 2 * M, ns=1) == INV
    assert rope(fn=lib.muse_rope_backward, qo=A + 128) == INV
    assert b"muse_rope_backward" in lib.muse_last_error()


def test_rope_frequencies(lib):
    def freq(out=A, rd=64, base=1e4, kind=0, factor=8.0, low=1.0, high=4.0, ctx=8192.0):
        return lib.muse_rope_frequencies(out, rd, base, kind, factor, low, high, ctx, None)

    assert freq(rd=0) == INV and freq(rd=7) == INV and freq(rd=258) == UNS
    assert freq(base=0.0) == INV and freq(base=float("nan")) == INV and freq(kind=9) == INV and freq(kind=-1) == INV
    for kind in (1, 2, 3, 4):
        assert freq(kind=kind, factor=0.0) == INV and freq(kind=kind, factor=float("inf")) == INV
    for kind in (3, 4):
        assert freq(kind=kind, low=4.0) == INV and freq(kind=kind, low=0.0) == INV and freq(kind=kind, ctx=0.0) == INV
        assert freq(kind=kind, high=float("inf")) == INV and freq(kind=kind, ctx=float("nan")) == INV
    assert freq(kind=4, base=1.0) == INV
    assert freq(out=None) == INV and freq(out=A + 4) == UNS


def test_expert_sort(lib):
    need = lib.muse_expert_sort_workspace_bytes(1 << 16, 64)
    assert need > 0 and lib.muse_expert_sort_workspace_bytes(64, 64) == 0
    assert lib.muse_expert_sort_workspace_bytes(-1, 64) == 0 and lib.muse_expert_sort_workspace_bytes(1 << 40, 64) == 0

    def sort(ids=A, kind=0, tokens=1 << 13, top_k=8, experts=64, off=A + M, row=A + 2 * M, slot=A + 3 * M, ws=A + 4 * M, n=need):
        return lib.muse_expert_sort(ids, kind, tokens, top_k, experts, off, row, slot, ws, n, None)

    assert sort(kind=2) == INV and sort(tokens=-1) == INV and sort(top_k=0) == INV and sort(experts=0) == INV
    assert sort(experts=1025) == UNS and sort(tokens=1 << 31, top_k=1) == UNS and sort(tokens=1 << 40) == UNS
    assert sort(ids=None) == INV and sort(off=None) == INV and sort(row=None) == INV and sort(slot=None) == INV
    assert sort(ws=None) == INV and sort(n=need - 1) == INV and sort(ws=A + 4 * M + 4) == UNS
    assert sort(ids=A + 2) == UNS and sort(ids=A + 4, kind=1) == UNS and sort(off=A + M + 1) == UNS and sort(slot=A + 3 * M + 2) == UNS
    assert sort(row=A) == INV and sort(slot=A + 2 * M) == INV and sort(off=A + 2 * M) == INV and sort(ws=A) == INV
    assert b"muse_expert_sort" in lib.muse_last_error()


def test_expert_rows(lib):
    def dispatch(x=A, rows=A + M, dt=BF16, tokens=8, hidden=64, k=2, n=16, xs=64, rs=64, row=A + 2 * M):
        return lib.muse_expert_dispatch(x, rows, dt, tokens, hidden, k, n, xs, rs, row, None)

    def combine(rows=A, y=A + M, dt=BF16, tokens=8, hidden=64, k=2, n=16, rs=64, ys=64, row=A + 2 * M, w=A + 3 * M):
        return lib.muse_expert_combine(rows, y, dt, tokens, hidden, k, n, rs, ys, row, w, None)

    def back(drows=A, dx=A + M, dt=BF16, tokens=8, hidden=64, k=2, n=16, rs=64, ys=64, row=A + 2 * M):
        return lib.muse_expert_dispatch_backward(drows, dx, dt, tokens, hidden, k, n, rs, ys, row, None)

    for fn in (dispatch, combine, back):
        assert fn(tokens=0) == 0
        assert fn(dt=3) == INV and fn(tokens=-1) == INV and fn(hidden=0) == INV and fn(k=0) == INV and fn(n=-1) == INV
        assert fn(hidden=60) == UNS and fn(hidden=40000) == UNS and fn(hidden=1 << 62) == UNS
        assert fn(tokens=1 << 30, k=2) == UNS and fn(n=1 << 31) == UNS
        assert fn(rs=32) == INV and fn(rs=68) == UNS and fn(row=None) == INV and fn(row=A + 2 * M + 2) == UNS
    assert dispatch(n=0) == 0
    assert dispatch(xs=32) == INV and dispatch(x=None) == INV and dispatch(rows=None) == INV and dispatch(x=A + 8) == UNS
    assert dispatch(rows=A) == INV and dispatch(rows=A + 2 * M) == INV and dispatch(xs=1 << 60) == UNS
    assert combine(ys=32) == INV and combine(y=None) == INV and combine(rows=None) == INV and combine(w=A + 3 * M + 2) == UNS
    assert combine(y=A) == INV and combine(y=A + 2 * M) == INV and combine(y=A + 3 * M) == INV
    assert back(dx=A + 64) == INV

    def bwd(rows=A, dy=A + M, drows=A + 2 * M, dt=BF16, tokens=8, hidden=64, k=2, n=16, rs=64, ys=64, ds=64, row=A + 3 * M,
            w=A + 4 * M, dw=A + 5 * M):
        return lib.muse_expert_combine_backward(rows, dy, drows, dt, tokens, hidden, k, n, rs, ys, ds, row, w, dw, None)

    assert bwd(tokens=0) == 0 and bwd(dt=9) == INV and bwd(hidden=4) == UNS
    assert bwd(rows=None) == INV and bwd(dy=None) == INV and bwd(drows=None) == INV and bwd(row=None) == INV
    assert bwd(rs=56) == INV and bwd(ys=8) == INV and bwd(ds=63) == INV and bwd(ds=65) == UNS and bwd(dy=A + M + 2) == UNS
    assert bwd(dw=A + 5 * M + 1) == UNS and bwd(w=A + 4 * M + 3) == UNS
    assert bwd(drows=A + 128) == INV and bwd(drows=A + M) == INV and bwd(drows=A + 4 * M) == INV
    assert bwd(dw=A + M) == INV and bwd(dw=A + 2 * M) == INV and bwd(dw=A + 4 * M + 4) == INV
    assert b"muse_expert_combine_backward" in lib.muse_last_error()
