"""The steps of a layer together, as a training step runs them: layer norm, rotary positions, the second layer norm, the
tokens to their experts, the per-expert norm, the experts (one scale and shift each: their products are no business of
this library), back to the tokens, blended into the residual stream; then the gradients the other way.

Every step is held to its own float64 formula on the very inputs it got, so the tolerances are those of the steps' own
tests; and the whole run gives the same bits launched back to back, with a wait after every call, and replayed from a
CUDA graph.
"""
import threading

import numpy as np
import pytest
import torch

import oracle
from gate_cores_b200 import _lib, cores
from gate_cores_b200.inputs import to_numpy
from oracle import steps

from .close64 import f64, near, same_bits
from .parity import check
from .test_gpu_expert import choices
from .test_gpu_layer_norm import BWD, FWD, PARAM

pytestmark = pytest.mark.gpu

B, S, HQ, HK, D, E, K = 3, 67, 4, 2, 64, 9, 3
H, T, EPS = HQ * D, B * S, 1e-5
EPS64 = float(np.float32(EPS))


def make(dt):
    g = torch.Generator().manual_seed(11)

    def n(*s, dtype=dt):
        return torch.randn(*s, generator=g).to(dtype).cuda()

    return {"x": n(T, H), "stream": n(T, H, dtype=torch.float32), "gain1": 1 + 0.2 * n(H, dtype=torch.float32),
            "bias1": n(H, dtype=torch.float32), "gain2": 1 + 0.2 * n(H, dtype=torch.float32), "key": n(T, HK * D),
            "inv_freq": cores.rope_frequencies(D, 1e4, "bands", 8.0, 1.0, 4.0, 64.0), "gains": 0.1 * n(E, H, dtype=torch.float32),
            "ids": choices(T, K, E, dropped=0.15).cuda(), "weights": torch.softmax(n(T, K, dtype=torch.float32), 1),
            "theta": n(H, dtype=torch.float32), "dstream": n(T, H, dtype=torch.float32), "dq": n(B, S, HQ, D)}


def run(s, wait=False):
    """Every intermediate result by name."""
    r = {}

    def step(**kw):
        r.update(kw)
        if wait:
            torch.cuda.synchronize()

    step(y1=cores.layer_norm(s["x"], s["gain1"], s["bias1"], eps=EPS))
    q, k = cores.rope(r["y1"].view(B, S, HQ, D), s["key"].view(B, S, HK, D), s["inv_freq"], pairing="half")
    step(q=q, k=k)
    step(y2=cores.layer_norm(r["q"].reshape(T, H), s["gain2"], eps=EPS))
    off, row, slot = cores.expert_sort(s["ids"], E)
    step(off=off, row=row, slot=slot)
    # rows that no slot names are the caller's: zeros here
    step(rows=cores.expert_dispatch(r["y2"], r["row"], out=torch.zeros(T * K, H, dtype=s["x"].dtype, device="cuda")))
    step(normed=cores.rms_norm_grouped(r["rows"], s["gains"], r["off"], 1.0, EPS))
    step(made=r["normed"] * 0.5)
    step(y=cores.expert_combine(r["made"], r["row"], s["weights"]))
    step(out=cores.residual_blend(s["stream"], r["y"], s["theta"]))
    dstream, dy, dtheta = cores.residual_backward(s["stream"], r["y"], s["dstream"], theta=s["theta"])
    step(d_stream=dstream, dy=dy, dtheta=dtheta)
    dmade, dw = cores.expert_combine_backward(r["made"], r["dy"], r["row"], s["weights"], drows=torch.zeros_like(r["made"]))
    step(dmade=dmade, dw=dw)
    step(drows=cores.rms_norm_backward(r["rows"], r["dmade"] * 0.5, None, eps=EPS)[0])  # without the gains
    step(dy2=cores.expert_dispatch_backward(r["drows"], r["row"]))
    dq, dgain2, dbias2 = cores.layer_norm_backward(r["q"].reshape(T, H), r["dy2"], s["gain2"], eps=EPS)
    step(dq=dq, dgain2=dgain2, dbias2=dbias2)
    step(dy1=cores.rope_backward((r["dq"].view(B, S, HQ, D) + s["dq"]), None, s["inv_freq"], pairing="half")[0])
    dx, dgain1, dbias1 = cores.layer_norm_backward(s["x"], r["dy1"].reshape(T, H), s["gain1"], eps=EPS)
    step(dx=dx, dgain1=dgain1, dbias1=dbias1)
    return r


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_each_step_on_what_it_got(cuda_ok, dt):
    s = make(dt)
    r = run(s)
    torch.cuda.synchronize()
    host = r["row"].cpu().numpy()
    pos = steps.rope_positions(T, S)
    near(r["y1"], steps.layer_norm(f64(s["x"]), f64(s["gain1"]), f64(s["bias1"]), 0.0, EPS64), FWD, "y1")
    near(r["q"].view(T, HQ, D), steps.rope(f64(r["y1"]).reshape(T, HQ, D), pos, f64(s["inv_freq"]), "half"), 8, "q")
    near(r["k"].view(T, HK, D), steps.rope(f64(s["key"]).reshape(T, HK, D), pos, f64(s["inv_freq"]), "half"), 8, "k")
    near(r["y2"], steps.layer_norm(f64(r["q"]).reshape(T, H), f64(s["gain2"]), None, 0.0, EPS64), FWD, "y2")
    for got, want in zip((r["off"], r["row"], r["slot"]), steps.expert_sort(s["ids"].cpu().numpy(), E)):
        assert np.array_equal(got.cpu().numpy(), want)
    kept = int(r["off"][-1])
    assert 0 < kept < T * K
    assert same_bits(r["rows"][:kept], r["y2"][r["slot"][:kept].long() // K]) and not r["rows"][kept:].any()
    check(to_numpy(r["normed"][:kept].cpu()),
          oracle.rms_norm_grouped(to_numpy(r["rows"][:kept].cpu()), s["gains"].cpu().numpy(), r["off"].cpu().numpy(), 1.0, EPS))
    near(r["y"], steps.expert_combine(f64(r["made"]), host, f64(s["weights"])), 2 * K, "y")
    (dmade, dmag), dw = steps.expert_combine_bwd(f64(r["made"]), f64(r["dy"]), host, f64(s["weights"]))
    near(r["dmade"][:kept], (dmade[:kept], dmag[:kept]), 1, "dmade")
    near(r["dw"], dw, 48, "dw")
    near(r["dy2"], steps.expert_combine(f64(r["drows"]), host), 2 * K, "dy2")
    for got, want, u in zip((r["dq"], r["dgain2"], r["dbias2"]),
                            steps.layer_norm_bwd(f64(r["q"]).reshape(T, H), f64(r["dy2"]), f64(s["gain2"]), 0.0, EPS64), (BWD, PARAM, PARAM)):
        near(got, want, u, "second norm")
    near(r["dy1"].reshape(T, HQ, D), steps.rope(f64(r["dq"].view(B, S, HQ, D) + s["dq"]).reshape(T, HQ, D), pos, f64(s["inv_freq"]),
                                                "half", backward=True), 8, "dy1")
    for got, want, u in zip((r["dx"], r["dgain1"], r["dbias1"]),
                            steps.layer_norm_bwd(f64(s["x"]), f64(r["dy1"]).reshape(T, H), f64(s["gain1"]), 0.0, EPS64), (BWD, PARAM, PARAM)):
        near(got, want, u, "first norm")
    assert _lib.muse_device_error() == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_back_to_back_waited_for_and_replayed(cuda_ok, dt):
    s = make(dt)
    want = run(s, wait=True)
    for _ in range(3):
        got = run(s)
        assert all(same_bits(want[n], got[n]) for n in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(s)
    for t in held.values():
        t.fill_(3)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(same_bits(want[n], held[n]) for n in want)


def test_two_runs_at_once(cuda_ok):
    a, b = make(torch.bfloat16), make(torch.float32)
    want = run(a), run(b)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i] = run(s)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(same_bits(w[n], g[n]) for n in w)


def test_the_default_stream_by_number(cuda_ok):
    s = make(torch.bfloat16)
    want = cores.layer_norm(s["x"], s["gain1"], s["bias1"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = cores.layer_norm(s["x"], s["gain1"], s["bias1"], stream=0)
        sort = cores.expert_sort(s["ids"], E, stream=0)
    torch.cuda.synchronize()
    assert same_bits(got, want)
    assert all(same_bits(x, y) for x, y in zip(sort, cores.expert_sort(s["ids"], E)))


def test_threads_of_one_program(cuda_ok):
    # every thread on a stream of its own; the calls run without the interpreter's lock, and an error reaches its thread
    x = torch.randn(700, 1024, device="cuda").bfloat16()
    ids = torch.rand(3000, 16, device="cuda").topk(4, 1).indices
    want = (cores.layer_norm(x), *cores.layer_norm_backward(x, x), *cores.expert_sort(ids, 16))
    torch.cuda.synchronize()
    wrong = []

    def work():
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                got = (cores.layer_norm(x, stream=s), *cores.layer_norm_backward(x, x, stream=s),
                       *cores.expert_sort(ids, 16, stream=s))
                s.synchronize()
                for a, b in zip(want, got):
                    assert (a is None and b is None) or torch.equal(a, b)
                with pytest.raises(_lib.MuseError, match="muse_layer_norm -> .*eps"):
                    cores.layer_norm(x, eps=-1.0, stream=s)
                with pytest.raises(_lib.MuseError, match="muse_expert_sort -> .*experts"):
                    cores.expert_sort(ids, 2000, stream=s)
        except BaseException as e:
            wrong.append(e)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
