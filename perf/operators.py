"""The measured cases of layer norm, rotary positions and the expert permutation.

`run` computes one pass of a case: with `own` true through gate_cores_b200, otherwise in elementary torch operations
in 32 bits (angles and far positions in 64), rounded once at the end.  `exact` is the operators' definition in 64 bits.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}
_EPS = 1e-6


def listed():
    return [
        # a decode step of 128 sequences: the pre-norm of one layer, latency counts
        {"name": "ln_decode_t128_h4096", "op": "layer_norm", "rows": 128, "hidden": 4096, "dtype": "bf16", "bias": True},
        # a vision tower's block norm over 16 images of 32x32 patches, 16 heads of 80
        {"name": "ln_vision_t16384_h1280", "op": "layer_norm", "rows": 16384, "hidden": 1280, "dtype": "bf16", "bias": True},
        # training, the prefill batch of 8192 tokens: input, gain and bias gradients
        {"name": "ln_bwd_t8192_h4096", "op": "layer_norm_backward", "rows": 8192, "hidden": 4096, "dtype": "bf16", "bias": True},
        # training in FP32 on a ragged batch with an odd row count and a width that is no power of two, no bias
        {"name": "ln_bwd_f32_t1999_h2600", "op": "layer_norm_backward", "rows": 1999, "hidden": 2600, "dtype": "f32", "bias": False},
        # a decode step of 128 sequences at far positions: halves paired, frequencies stretched by bands
        {"name": "rope_decode_t128_half", "op": "rope", "dtype": "bf16", "layout": "explicit", "batch": 128, "seqlen": 1, "hq": 32,
         "hk": 8, "head_dim": 128, "rotary_dim": 128, "pairing": "half", "scaling": "bands", "fused": True},
        # sixteen packed documents, about 70 thousand tokens: adjacent pairs, half of each head rotated
        {"name": "rope_thd16_partial", "op": "rope", "dtype": "bf16", "layout": "thd", "batch": 16, "seqlen": 8192, "hq": 40,
         "hk": 8, "head_dim": 128, "rotary_dim": 64, "pairing": "interleaved", "scaling": "none", "fused": False},
        # training, the gradient through the prefill batch's rotation in FP32: halves paired, frequencies ramped
        {"name": "rope_bwd_f32_t8192_half", "op": "rope_backward", "dtype": "f32", "layout": "bshd", "batch": 2, "seqlen": 4096,
         "hq": 32, "hk": 8, "head_dim": 128, "rotary_dim": 128, "pairing": "half", "scaling": "ramp", "fused": False},
        # a decode step of 128 sequences through 64 experts, 8 for each token: sort, rows out to the experts, rows back
        {"name": "experts_decode_t128", "op": "experts", "dtype": "bf16", "tokens": 128, "hidden": 4096, "top_k": 8, "experts": 64,
         "dropped": 0.0},
        # the sort alone for a packed batch of 80251 tokens
        {"name": "expert_sort_t80251_k8", "op": "expert_sort", "tokens": 80251, "top_k": 8, "experts": 64, "dropped": 0.0},
        # the prefill batch through 64 experts, 8 for each token, some choices dropped by the router
        {"name": "experts_t8192_h4096_k8", "op": "experts", "dtype": "bf16", "tokens": 8192, "hidden": 4096, "top_k": 8,
         "experts": 64, "dropped": 0.05},
        # training on the prefill batch: gradients of the rows, the weights and the tokens, 4 experts for each token
        {"name": "experts_bwd_t8192_h5120_k4", "op": "experts_backward", "dtype": "bf16", "tokens": 8192, "hidden": 5120, "top_k": 4,
         "experts": 64, "dropped": 0.0},
        # training in FP32 on a small ragged batch, 2 experts for each token, some choices dropped
        {"name": "experts_bwd_f32_t777_h1000", "op": "experts_backward", "dtype": "f32", "tokens": 777, "hidden": 1000, "top_k": 2,
         "experts": 8, "dropped": 0.1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_backward", "rope", "rope_backward", "expert_sort", "experts", "experts_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("layer_norm", "layer_norm_backward"):
        hidden = 8 * _log(rng, 8, 1024 if dtype == "bf16" else 512)
        rows = min(_log(rng, 1, 32768), 8192 * 8192 // hidden)
        return {"op": op, "rows": rows, "hidden": hidden, "dtype": dtype, "bias": rng.random() < 0.7}
    if op in ("rope", "rope_backward"):
        d = rng.choice([64, 80, 96, 128, 128, 256] if dtype == "bf16" else [64, 80, 96, 128])
        hk = rng.choice([1, 2, 4, 5, 8])
        layout = rng.choice(["bshd", "thd", "explicit"])
        batch = _log(rng, 1, 64)
        return {"op": op, "dtype": dtype, "layout": layout, "batch": batch, "seqlen": _log(rng, 1, 32768 // batch),
                "hq": hk * rng.choice([1, 2, 4, 5, 8]), "hk": hk, "head_dim": d, "rotary_dim": d // rng.choice([1, 1, 2, 4]),
                "pairing": rng.choice(["half", "interleaved"]), "scaling": rng.choice(["none", "linear", "base", "bands", "ramp"]),
                "fused": rng.random() < 0.5}
    top_k = rng.choice([1, 2, 3, 4, 6, 8])
    experts = max(top_k, _log(rng, 4, 512))
    dropped = rng.choice([0.0, 0.0, 0.1])
    if op == "expert_sort":
        return {"op": op, "tokens": _log(rng, 1, 80251), "top_k": top_k, "experts": experts, "dropped": dropped}
    hidden = 8 * _log(rng, 8, 1024)
    tokens = min(_log(rng, 1, 16384), 8192 * 8 * 4096 // (hidden * top_k * (_ES[dtype] // 2)))
    return {"op": op, "dtype": dtype, "tokens": tokens, "hidden": hidden, "top_k": top_k, "experts": experts, "dropped": dropped}


def work(case):
    op = case["op"]
    if op in ("layer_norm", "layer_norm_backward"):
        n, e, h = case["rows"] * case["hidden"], _ES[case["dtype"]], case["hidden"]
        if op == "layer_norm":
            return {"bytes": 2 * n * e + 4 * h * (2 if case["bias"] else 1), "flops": 8 * n}
        return {"bytes": 3 * n * e + 4 * h * (3 if case["bias"] else 2), "flops": 15 * n}
    if op in ("rope", "rope_backward"):
        tokens = _tokens(case)
        n = tokens * (case["hq"] + case["hk"])
        more = 4 * tokens if case["layout"] == "explicit" else 0
        return {"bytes": 2 * n * case["head_dim"] * _ES[case["dtype"]] + more, "flops": 3 * n * case["rotary_dim"]}
    slots = case["tokens"] * case["top_k"]
    sort = 3 * 4 * slots + 4 * (case["experts"] + 1)  # the choices in, the permutation and its inverse out
    if op == "expert_sort":
        return {"bytes": sort, "flops": slots}
    one = case["tokens"] * case["hidden"] * _ES[case["dtype"]]  # a token's row each
    if op == "experts":  # every token in, its rows out; the rows in (as many), every token out, with the weights
        return {"bytes": sort + 2 * (1 + case["top_k"]) * one + 4 * slots, "flops": 2 * slots * case["hidden"]}
    # the tokens' gradients and the rows in, the rows' gradients out; rows' gradients in, the tokens' out; weights in and out
    return {"bytes": (2 + 3 * case["top_k"]) * one + 3 * 4 * slots, "flops": 4 * slots * case["hidden"]}


def _lengths(case):
    """The documents of a packed batch: lengths between a sixteenth of the longest and the longest, the same for every seed."""
    n, longest = case["batch"], case["seqlen"]
    return [max(1, longest - (longest * 15 // 16) * ((7 * i) % n) // max(1, n - 1)) for i in range(n)]


def _tokens(case):
    return sum(_lengths(case)) if case["layout"] == "thd" else case["batch"] * case["seqlen"]


def _frequencies(case):
    """The plan that a model keeps: radians per position of each pair, in 64 bits, and the factor on cos and sin."""
    rd, base = case["rotary_dim"], 5.0e5
    i = torch.arange(rd // 2, dtype=torch.float64)
    kind, factor, context = case["scaling"], 8.0, 8192.0
    if kind == "base" and rd > 2:
        base *= factor ** (rd / (rd - 2))
    f = base ** (-2.0 * i / rd)
    if kind == "linear":
        f = f / factor
    if kind == "bands":  # long waves are stretched, short ones stay, between them a blend by waves in the context
        mix = ((context * f / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = f * (mix + (1 - mix) / factor)
    if kind == "ramp":  # the same between two indexes: those of pairs that turn 32 times and once in the context
        low, high = (rd * math.log(context / (2 * math.pi * t)) / (2 * math.log(base)) for t in (32.0, 1.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), rd - 1)
        mix = 1 - ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f * (mix + (1 - mix) / factor)
    return f, (0.1 * math.log(factor) + 1.0 if kind == "ramp" else 1.0)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    op = case["op"]
    if op in ("layer_norm", "layer_norm_backward"):
        dt, rows, hidden = _DT[case["dtype"]], case["rows"], case["hidden"]
        shift = 0.5 * normal(rows, 1)  # rows with means of their own, as a residual stream has them
        s = {"op": op, "x": (normal(rows, hidden) + shift).to(dt), "gain": 0.5 + torch.rand(hidden, generator=g, device=dev),
             "bias": normal(hidden) if case["bias"] else None}
        if op == "layer_norm_backward":
            s["dy"] = normal(rows, hidden, dtype=dt)
        return s
    if op in ("rope", "rope_backward"):
        dt, tokens, d = _DT[case["dtype"]], _tokens(case), case["head_dim"]
        hq, hk = case["hq"], case["hk"]
        if case["fused"]:  # views into one projection of Q, K and V
            both = normal(tokens, hq + 2 * hk, d, dtype=dt)
            q, k = both[:, :hq], both[:, hq:hq + hk]
        else:
            q, k = normal(tokens, hq, d, dtype=dt), normal(tokens, hk, d, dtype=dt)
        f, scale = _frequencies(case)
        s = {"op": op, "q": q, "k": k, "inv_freq": f.to(dev), "scale": scale, "pairing": case["pairing"], "layout": case["layout"],
             "positions": None, "cu_seqlens": None}
        if case["layout"] == "explicit":
            s["positions"] = torch.randint(0, 131072, (tokens,), generator=g, device=dev, dtype=torch.int32)
        elif case["layout"] == "thd":
            cu = torch.tensor([0] + _lengths(case)).cumsum(0)
            s["cu_seqlens"] = cu.to(torch.int32).to(dev)
        else:
            s["q"], s["k"] = (t.unflatten(0, (case["batch"], case["seqlen"])) for t in (q, k))
        return s
    tokens, top_k, experts = case["tokens"], case["top_k"], case["experts"]
    # a router's choices: experts of uneven popularity, top_k different ones for each token
    score = torch.rand(tokens, experts, generator=g, device=dev) ** (0.25 + 1.5 * torch.rand(experts, generator=g, device=dev))
    ids = score.topk(top_k, dim=1).indices.to(torch.int32)
    if case["dropped"]:
        ids = torch.where(torch.rand(tokens, top_k, generator=g, device=dev) < case["dropped"], torch.full_like(ids, -1), ids)
    s = {"op": op, "ids": ids, "experts": experts}
    if op == "expert_sort":
        return s
    dt, hidden = _DT[case["dtype"]], case["hidden"]
    s["weights"] = torch.softmax(normal(tokens, top_k), 1)
    s["rows"] = torch.zeros(tokens * top_k, hidden, dtype=dt, device=dev)  # a buffer that the program keeps
    s["outputs"] = normal(tokens * top_k, hidden, dtype=dt)  # what the experts made of the rows
    if op == "experts":
        s["x"] = normal(tokens, hidden, dtype=dt)
    else:
        s["dy"] = normal(tokens, hidden, dtype=dt)
        s["row_of_slot"] = _sorted(ids, experts)[1]  # kept from the forward pass
    return s


# ---- the plain forms


def _sorted(ids, experts):
    """(group_offsets, row_of_slot, slot_of_row): slots in the order of their experts, equal ones in their own; dropped slots have row -1."""
    flat = ids.reshape(-1).to(torch.int64)
    kept = (flat >= 0) & (flat < experts)
    order = torch.sort(torch.where(kept, flat, experts), stable=True).indices
    place = torch.arange(flat.numel(), device=flat.device)
    rank = torch.empty_like(place)
    rank[order] = place
    edges = torch.arange(experts + 1, device=flat.device)
    offsets = torch.searchsorted(torch.where(kept, flat, experts)[order], edges)
    return (offsets.to(torch.int32), torch.where(kept, rank, -1).to(torch.int32).view(ids.shape),
            torch.where(place < offsets[-1], order, -1).to(torch.int32))


def _plain_layer_norm(s):
    x = s["x"].float()
    c = x - x.mean(-1, keepdim=True)
    y = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + _EPS) * s["gain"]
    return (y if s["bias"] is None else y + s["bias"]).to(s["x"].dtype)


def _plain_layer_norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    c = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((c * c).mean(-1, keepdim=True) + _EPS)
    n, g = c * r, dy * s["gain"]
    dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    grads = [dx.to(s["x"].dtype), (dy * n).sum(0)]
    return grads if s["bias"] is None else grads + [dy.sum(0)]


def _positions(s):
    if s["positions"] is not None:
        return s["positions"].to(torch.int64)
    if s["cu_seqlens"] is not None:
        t = torch.arange(s["q"].shape[0], device=s["q"].device)
        cu = s["cu_seqlens"].to(torch.int64)
        return t - cu[torch.searchsorted(cu, t, right=True) - 1]
    return torch.arange(s["q"].shape[1], device=s["q"].device).expand(s["q"].shape[:2])


def _plain_rope(s, sign):
    angle = (_positions(s).double()[..., None] * s["inv_freq"])[..., None, :]
    c, n = (torch.cos(angle) * s["scale"]).float(), (torch.sin(angle) * (sign * s["scale"])).float()
    half = s["inv_freq"].numel()

    def turn(t):
        u = t.float()
        rot, rest = u[..., :2 * half], u[..., 2 * half:]
        if s["pairing"] == "half":
            a, b = rot[..., :half], rot[..., half:]
            rot = torch.cat([a * c - b * n, a * n + b * c], -1)
        else:
            a, b = rot[..., 0::2], rot[..., 1::2]
            rot = torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)
        return torch.cat([rot, rest], -1).to(t.dtype)

    return [turn(s["q"]), turn(s["k"])]


def _plain_experts(s):
    offsets, row_of_slot, slot_of_row = _sorted(s["ids"], s["experts"])
    tokens, top_k = s["ids"].shape
    kept = (slot_of_row >= 0)[:, None]
    # the buffer's rows behind the last group stay as they are
    rows = torch.where(kept, s["x"][(slot_of_row // top_k).clamp(min=0).long()], s["rows"])
    w = torch.where(row_of_slot >= 0, s["weights"], 0.0)
    y = (s["outputs"][row_of_slot.clamp(min=0).long()].float() * w[..., None]).sum(1)
    return [offsets, row_of_slot, slot_of_row, rows, y.to(s["x"].dtype)]


def _plain_experts_backward(s):
    row, w = s["row_of_slot"], s["weights"]
    kept = row >= 0
    at, dy = row.clamp(min=0).long(), s["dy"].float()
    drows = s["rows"].clone()
    drows[row[kept].long()] = (w[..., None] * dy[:, None]).to(drows.dtype)[kept]
    dw = torch.where(kept, (s["outputs"][at].float() * dy[:, None]).sum(-1), 0.0)
    dx = torch.where(kept[..., None], drows[at].float(), 0.0).sum(1)
    return [drows, dw, dx.to(drows.dtype)]


def run(s):
    op = s["op"]
    if own:
        return _own(s)
    if op == "layer_norm":
        return _plain_layer_norm(s)
    if op == "layer_norm_backward":
        return _plain_layer_norm_backward(s)
    if op in ("rope", "rope_backward"):
        return _plain_rope(s, 1.0 if op == "rope" else -1.0)
    if op == "expert_sort":
        return list(_sorted(s["ids"], s["experts"]))
    return _plain_experts(s) if op == "experts" else _plain_experts_backward(s)


def _own(s):
    from gate_cores_b200 import cores

    op = s["op"]
    if op == "layer_norm":
        return cores.layer_norm(s["x"], s["gain"], s["bias"], eps=_EPS)
    if op == "layer_norm_backward":
        dx, dgain, dbias = cores.layer_norm_backward(s["x"], s["dy"], s["gain"], eps=_EPS, want_dbias=s["bias"] is not None)
        return [dx, dgain] if dbias is None else [dx, dgain, dbias]
    if op in ("rope", "rope_backward"):
        turn = cores.rope if op == "rope" else cores.rope_backward
        return list(turn(s["q"], s["k"], s["inv_freq"], positions=s["positions"], cu_seqlens=s["cu_seqlens"], pairing=s["pairing"],
                         attention_scale=s["scale"]))
    if op == "expert_sort":
        return list(cores.expert_sort(s["ids"], s["experts"]))
    if op == "experts":
        offsets, row_of_slot, slot_of_row = cores.expert_sort(s["ids"], s["experts"])
        rows = cores.expert_dispatch(s["x"], row_of_slot, out=s["rows"])
        return [offsets, row_of_slot, slot_of_row, rows, cores.expert_combine(s["outputs"], row_of_slot, s["weights"])]
    drows, dw = cores.expert_combine_backward(s["outputs"], s["dy"], s["row_of_slot"], s["weights"], drows=s["rows"])
    return [drows, dw, cores.expert_dispatch_backward(drows, s["row_of_slot"])]


# ---- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "expert_sort":
        return None
    if op in ("layer_norm", "layer_norm_backward"):
        x, w = s["x"].double(), s["gain"].double()
        h = x.shape[1]
        mean = x.sum(1) / h
        dev = torch.sqrt(((x - mean[:, None]) ** 2).sum(1) / h + _EPS)
        n = (x - mean[:, None]) / dev[:, None]
        if op == "layer_norm":
            return n * w + (0.0 if s["bias"] is None else s["bias"].double())
        dy = s["dy"].double()
        g = dy * w
        # the Jacobian of a row: (I - 1 1'/h - n n'/h) / dev
        dx = (g - g.sum(1, keepdim=True) / h - n * ((n * g).sum(1, keepdim=True) / h)) / dev[:, None]
        grads = [dx, torch.einsum("rh,rh->h", dy, n)]
        return grads if s["bias"] is None else grads + [dy.sum(0)]
    if op in ("rope", "rope_backward"):
        if case["layout"] == "explicit":
            at = s["positions"].double()
        elif case["layout"] == "thd":
            at = torch.cat([torch.arange(n) for n in _lengths(case)]).double().cuda()
        else:
            at = torch.arange(case["seqlen"]).double().cuda().repeat(case["batch"])
        turn = at[:, None] * s["inv_freq"] * (1.0 if op == "rope" else -1.0)
        unit = torch.polar(torch.full_like(turn, s["scale"]), turn)[:, None, :]
        rd, outs = case["rotary_dim"], []
        for t in (s["q"], s["k"]):
            u = t.double().reshape(at.numel(), t.shape[-2], t.shape[-1])
            v = u[..., :rd].contiguous()
            if case["pairing"] == "half":
                z = torch.complex(v[..., :rd // 2], v[..., rd // 2:]) * unit
                v = torch.cat([z.real, z.imag], -1)
            else:
                v = torch.view_as_real(torch.view_as_complex(v.unflatten(-1, (rd // 2, 2))) * unit).flatten(-2)
            outs.append(torch.cat([v, u[..., rd:]], -1).reshape(t.shape))
        return outs
    w = s["weights"].double()
    ids = s["ids"]
    if op == "experts":
        x, outputs = s["x"].double(), s["outputs"].double()
        rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device=x.device)
        chosen = [(ids.reshape(-1) == e).nonzero()[:, 0] for e in range(s["experts"])]
        slots = torch.cat(chosen)
        token = slots // ids.shape[1]
        rows[:token.numel()] = x[token]
        y = torch.zeros_like(x).index_add_(0, token, outputs[:token.numel()] * w.reshape(-1)[slots, None])
        return [None, None, None, rows, y]
    dy, outputs, row = s["dy"].double(), s["outputs"].double(), s["row_of_slot"]
    drows = torch.zeros_like(outputs)
    dw = torch.zeros_like(w)
    dx = torch.zeros_like(dy)
    for j in range(ids.shape[1]):
        t = (row[:, j] >= 0).nonzero()[:, 0]
        r = row[t, j].long()
        grad = w[t, j, None] * dy[t]
        drows[r] = grad
        dw[t, j] = torch.einsum("th,th->t", dy[t], outputs[r])
        dx[t] += grad.to(s["rows"].dtype).double()  # the rows' gradients are handed on in their type
    return [drows, dw, dx]
