"""Measured cases of the operators beside the expert FFN that a model with its own
expert products, a shared expert or dense blocks needs, and that training needs:
the rows of the tokens in expert order and back (with the routing weights, and the
gradients of both), layer norm with its gradients, and the matrix product with
bias, activation (gated or not) and residual in its epilogue.

``run`` computes a case in its plain form (elementary torch operations in fp32,
rounded once at the end) or, where ``own`` is set, through this library's entry
points. Sizes follow the library's workloads (hidden 4096 and 7168, intermediate
2048, 64 and 128 experts, top-8, batches of 16 and 4096 tokens) or are generic.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-5
_ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ---------------------------------------------------------------- cases ---

def _rows(op, T, k, H, E, local, block_m, dtype="bf16", rows_dtype=None):
    """Tokens in expert order: T tokens of k slots each, E experts of which the
    first ``local`` are here, runs padded to block_m; ``dtype`` of the tokens,
    ``rows_dtype`` of the rows in expert order (dispatch: the same)."""
    return dict(op=op, T=T, k=k, H=H, E=E, local=local, block_m=block_m, dtype=dtype,
                rows_dtype=rows_dtype or dtype)


def _norm(op, T, H, dtype="bf16", residual=True, affine=True):
    return dict(op=op, T=T, H=H, dtype=dtype, residual=residual, affine=affine)


def _linear(T, N, K, act="none", gated=False, bias=False, residual=False, dtype="bf16",
            out_dtype=None):
    return dict(op="linear", T=T, N=N, K=K, act=act, gated=gated, bias=bias, residual=residual,
                dtype=dtype, out_dtype=out_dtype or dtype)


def listed():
    return [
        # a decode step's tokens laid out for a grouped product over all experts: latency
        dict(_rows("dispatch", 16, 8, 4096, 64, 64, 16), name="dispatch_decode_16x8x4096"),
        # the same for a prompt or a training batch: one read, eight copies of every token
        dict(_rows("dispatch", 4096, 8, 4096, 128, 128, 128),
             name="dispatch_prefill_4096x8x4096"),
        # the way back with the routing weights: bound by the experts' rows
        dict(_rows("combine", 4096, 8, 4096, 128, 128, 128), name="combine_prefill_4096x8x4096"),
        # gradient of the dispatch on an expert-parallel rank that holds a quarter of the experts:
        # most slots are elsewhere, some tokens have none here
        dict(_rows("dispatch_backward", 1021, 6, 2048, 64, 16, 64),
             name="dispatch_backward_shard_1021x6x2048"),
        # gradient of the combine of a training batch: the largest case of the rows
        dict(_rows("combine_backward", 4096, 8, 4096, 128, 128, 128),
             name="combine_backward_4096x8x4096"),
        # the same in fp32, unpadded runs, odd sizes: a small model's micro-batch
        dict(_rows("combine_backward", 250, 4, 1030, 60, 60, 1, "f32"),
             name="combine_backward_f32_250x4x1030"),
        # a decode step's residual add and layer norm: latency
        dict(_norm("layer_norm", 16, 4096), name="layer_norm_decode_16x4096"),
        # its gradients for a training batch, the residual's among them: the activations once,
        # and sums over all rows for the weight and the bias
        dict(_norm("layer_norm_backward", 4096, 4096), name="layer_norm_backward_4096x4096"),
        # forward and backward in fp32 over rows of an odd length
        dict(_norm("layer_norm_train", 777, 1031, "f32", residual=False),
             name="layer_norm_train_f32_777x1031"),
        # gate|up projection of the shared expert in a decode step: bound by the weights
        dict(_linear(16, 2048, 7168, "silu", gated=True), name="linear_decode_16x2048x7168_gated"),
        # up projection of a dense block, biased, a ragged batch and an odd width
        dict(_linear(509, 4100, 4096, "gelu_tanh", bias=True), name="linear_509x4100x4096_gelu"),
        # a square projection of a prompt with bias and the residual added in the epilogue:
        # bound by the matrix cores
        dict(_linear(4096, 7168, 4096, bias=True, residual=True),
             name="linear_prefill_4096x7168x4096"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _length(rng, lo, hi):
    """A row length: mostly a multiple of 8, now and then any."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.2 else max(8, n // 8 * 8)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("dispatch", "combine", "dispatch_backward", "combine_backward",
                         "layer_norm", "layer_norm_backward", "layer_norm_train", "linear",
                         "linear", "linear", "linear"))
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        if op == "linear":
            gated = rng.random() < 0.4
            c = _linear(_log(rng, 1, 8192), _log(rng, 64, 8192),
                        max(64, _log(rng, 64, 8192) // 8 * 8), rng.choice(_ACTS), gated,
                        rng.random() < 0.5, rng.random() < 0.4, dtype,
                        rng.choice((dtype, "f32")))
        elif op.startswith("layer_norm"):
            c = _norm(op, _log(rng, 1, 8192), _length(rng, 64, 8192), dtype, rng.random() < 0.6,
                      rng.random() < 0.8)
        else:
            E = rng.choice((8, 60, 64, 128, 160, 256))
            c = _rows(op, _log(rng, 1, 4096), rng.choice((1, 2, 4, 6, 8)),
                      _length(rng, 64, 8192), E, rng.choice((E, E, E // 4)),
                      rng.choice((1, 16, 64, 128)), dtype,
                      rng.choice((dtype, "f32")) if op.startswith("combine") else dtype)
        if _cost(c) <= most:
            return c


def work(case):
    c = case
    if c["op"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        n = 2 * N if c["gated"] else N
        b, bo = _BYTES[c["dtype"]], _BYTES[c["out_dtype"]]
        byt = (T + n) * K * b + T * N * bo * (2 if c["residual"] else 1) + 4 * n * c["bias"]
        return {"bytes": byt, "flops": 2 * T * n * K}
    if c["op"].startswith("layer_norm"):
        n, b = c["T"] * c["H"], _BYTES[c["dtype"]]
        fwd, bwd = 2 + 2 * c["residual"], 3 + 2 * c["residual"]
        vec = 4 * c["H"]
        streams, vecs, flops = {
            "layer_norm": (fwd, 2 * c["affine"], 8),
            "layer_norm_backward": (bwd, 2 * c["affine"] + 1, 14),
            "layer_norm_train": (fwd + bwd, 4 * c["affine"] + 1, 22)}[c["op"]]
        return {"bytes": n * b * streams + vec * vecs, "flops": flops * n}
    S = c["T"] * c["k"]
    slots = S * c["local"] / c["E"]
    used = c["local"] * (1 - (1 - 1 / c["E"]) ** S)   # experts with a run
    padded = slots + used * (c["block_m"] - 1) / 2
    tok = c["T"] * c["H"] * _BYTES[c["dtype"]]
    row = c["H"] * _BYTES[c["rows_dtype"]]
    if c["op"] == "dispatch":
        return {"bytes": tok + padded * row + 8 * S + 4 * padded, "flops": 0}
    if c["op"] == "combine":
        return {"bytes": tok + slots * row + 8 * S, "flops": 2 * slots * c["H"]}
    if c["op"] == "dispatch_backward":
        return {"bytes": tok + slots * row + 4 * S, "flops": slots * c["H"]}
    return {"bytes": tok + (slots + padded) * row + 12 * S + 4 * padded,
            "flops": 3 * slots * c["H"]}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / (200 if case.get("dtype") == "bf16" else 25))


# --------------------------------------------------------------- inputs ---

def _lists(ids, E, block_m):
    """The slots ordered by expert, runs padded to block_m with the number of slots:
    (sorted_ids, num_padded), as a layer has them from the alignment."""
    S = ids.numel()
    flat = ids.reshape(-1).long()
    cap = (S + min(E, S) * (block_m - 1) + block_m - 1) // block_m * block_m
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    count = torch.bincount(key, minlength=E + 1)
    padded = (count[:E] + block_m - 1) // block_m * block_m
    ends = torch.cumsum(padded, 0)
    first = torch.cumsum(count, 0) - count
    k = key[order]
    at = (ends - padded)[k.clamp(max=E - 1)] + torch.arange(S, device=ids.device) - first[k]
    sid = torch.full((cap + 1,), S, dtype=torch.int32, device=ids.device)
    sid[torch.where(k < E, at, cap)] = torch.where(k < E, order, S).int()
    return sid[:cap].contiguous(), ends[-1:].int()


def _where(ids, E, sorted_ids, num_padded):
    """live [R]: the rows that hold a slot; at [T, k]: every slot's row, -1 for none."""
    S, R = ids.numel(), sorted_ids.numel()
    p = torch.arange(R, device=ids.device)
    live = (p < num_padded) & (sorted_ids < S)
    at = torch.full((S + 1,), -1, dtype=torch.int32, device=ids.device)
    at[torch.where(live, sorted_ids, S).long()] = p.int()
    return live, at[:S].view(ids.shape)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(1 + seed)

    def normal(*shape, dtype="f32", std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(_DT[dtype])

    s = {"case": c}
    if c["op"] == "linear":
        n = 2 * c["N"] if c["gated"] else c["N"]
        s["x"] = normal(c["T"], c["K"], dtype=c["dtype"])
        s["w"] = normal(n, c["K"], dtype=c["dtype"], std=c["K"] ** -0.5)
        s["bias"] = normal(n, std=0.3) if c["bias"] else None
        s["residual"] = (normal(c["T"], c["N"], dtype=c["out_dtype"], std=4.0)
                         if c["residual"] else None)
        return s
    if c["op"].startswith("layer_norm"):
        T, H = c["T"], c["H"]
        # a residual stream with a few channels far larger than the others
        s["x"] = normal(T, H, dtype=c["dtype"])
        big = 4.0 * torch.ones(H, device="cuda")
        big[torch.randint(0, H, (3,), generator=g, device="cuda")] = 40.0
        stream = (torch.randn((T, H), generator=g, device="cuda") * big + 0.5).to(_DT[c["dtype"]])
        s["residual"] = stream if c["residual"] else None
        s["weight"] = 1 + 0.1 * normal(H) if c["affine"] else None
        s["bias"] = 0.1 * normal(H) if c["affine"] else None
        s["alpha"] = 0.75
        if c["op"] != "layer_norm":
            s["dout"] = normal(T, H, dtype=c["dtype"], std=0.02)
            s["dsum"] = normal(T, H, dtype=c["dtype"], std=0.02) if c["residual"] else None
        if c["op"] == "layer_norm_backward":
            s["sum"] = stream      # what the forward pass left
        return s
    T, k, H, E, local = c["T"], c["k"], c["H"], c["E"], c["local"]
    # softmax over logits with popular experts; ids from `local` on are another rank's
    logits = normal(T, E) + normal(E)
    p, ids = torch.topk(torch.softmax(logits, 1), k, dim=1)
    s["ids"], s["weights"] = ids.int().contiguous(), p.contiguous()
    s["sorted_ids"], s["num_padded"] = _lists(s["ids"], local, c["block_m"])
    R = s["sorted_ids"].numel()
    live, s["slot_rows"] = _where(s["ids"], local, s["sorted_ids"], s["num_padded"])
    if c["op"] == "dispatch":
        s["x"] = normal(T, H, dtype=c["dtype"])
    if c["op"] == "combine_backward":
        s["dout"] = normal(T, H, dtype=c["dtype"], std=0.02)
    if c["op"] != "dispatch":
        # what the experts' products give; the rows of no slot hold anything
        s["rows"] = normal(R, H, dtype=c["rows_dtype"])
        s["rows"][~live] = float("nan")
    if c["op"] in ("dispatch", "combine_backward"):
        # rows behind the last run are left as they are
        s["out"] = torch.zeros((R, H), dtype=_DT[c["rows_dtype"]], device="cuda")
    return s


# ------------------------------------------------------------------ run ---

def run(state):
    return _RUN[state["case"]["op"]](state)


def _run_dispatch(s):
    c = s["case"]
    if own:
        import moe_expert_ffn_router_amd as moe
        return list(moe.dispatch(s["x"], s["ids"], c["local"], s["sorted_ids"], s["num_padded"],
                                 out=s["out"]))
    S = s["ids"].numel()
    live, at = _where(s["ids"], c["local"], s["sorted_ids"], s["num_padded"])
    rows = s["x"][s["sorted_ids"].long().clamp(max=S - 1) // c["k"]]
    rows[~live] = 0
    return [rows, at]


def _gathered(s):
    """The rows of every token's slots in fp32, zeros where a slot has none: [T, k, H]."""
    here = (s["slot_rows"] >= 0).unsqueeze(-1)
    return torch.where(here, s["rows"][s["slot_rows"].long().clamp(min=0)].float(), 0.0)


def _run_combine(s):
    c = s["case"]
    if own:
        import moe_expert_ffn_router_amd as moe
        return [moe.combine(s["rows"], s["slot_rows"], s["weights"], dtype=_DT[c["dtype"]])]
    return [(_gathered(s) * s["weights"].unsqueeze(-1)).sum(1).to(_DT[c["dtype"]])]


def _run_dispatch_backward(s):
    if own:
        import moe_expert_ffn_router_amd as moe
        return [moe.dispatch_backward(s["rows"], s["slot_rows"])]
    return [_gathered(s).sum(1).to(_DT[s["case"]["dtype"]])]


def _run_combine_backward(s):
    c = s["case"]
    if own:
        import moe_expert_ffn_router_amd as moe
        return list(moe.combine_backward(s["dout"], s["rows"], s["slot_rows"], s["weights"],
                                         s["sorted_ids"], s["num_padded"], drows=s["out"]))
    S = s["ids"].numel()
    live, _ = _where(s["ids"], c["local"], s["sorted_ids"], s["num_padded"])
    slot = s["sorted_ids"].long().clamp(max=S - 1)
    drows = s["dout"].float()[slot // c["k"]] * s["weights"].reshape(-1)[slot].unsqueeze(-1)
    drows = torch.where(live.unsqueeze(-1), drows, 0.0).to(_DT[c["rows_dtype"]])
    dweights = (_gathered(s) * s["dout"].float().unsqueeze(1)).sum(-1)
    return [drows, dweights]


def _norm_forward(s):
    v = s["alpha"] * s["x"].float()
    if s["residual"] is not None:
        v = s["residual"].float() + v
    d = v - v.mean(-1, keepdim=True)
    out = d * torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    if s["weight"] is not None:
        out = out * s["weight"] + s["bias"]
    return out.to(s["x"].dtype), v.to(s["x"].dtype)


def _norm_backward(s, total):
    v, dout = total.float(), s["dout"].float()
    d = v - v.mean(-1, keepdim=True)
    inv = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    unit = d * inv
    g = dout if s["weight"] is None else dout * s["weight"]
    ds = (g - g.mean(-1, keepdim=True) - unit * (g * unit).mean(-1, keepdim=True)) * inv
    if s["dsum"] is not None:
        ds = ds + s["dsum"].float()
    out = [(s["alpha"] * ds).to(total.dtype)]
    if s["dsum"] is not None:
        out.append(ds.to(total.dtype))
    if s["weight"] is not None:
        out.append((dout * unit).sum(0))
    return out + [dout.sum(0)]


def _own_backward(s, total):
    import moe_expert_ffn_router_amd as moe
    grads = moe.layer_norm_backward(s["dout"], total, s["weight"], dresidual_out=s["dsum"],
                                    alpha=s["alpha"], eps=EPS)
    return [t for t in grads if t is not None]


def _own_forward(s, residual_out=None):
    import moe_expert_ffn_router_amd as moe
    return moe.layer_norm(s["x"], s["weight"], s["bias"], residual=s["residual"],
                          alpha=s["alpha"], eps=EPS, residual_out=residual_out)


def _run_layer_norm(s):
    out, total = _own_forward(s) if own else _norm_forward(s)
    return [out] if s["residual"] is None else [out, total]


def _run_layer_norm_backward(s):
    return _own_backward(s, s["sum"]) if own else _norm_backward(s, s["sum"])


def _run_layer_norm_train(s):
    if own:
        keep = torch.empty_like(s["x"]) if s["residual"] is None else None
        out, total = _own_forward(s, keep)
        return [out, total] + _own_backward(s, total)
    out, total = _norm_forward(s)
    return [out, total] + _norm_backward(s, total)


def _act(name, v):
    if name == "relu":
        return torch.where(v < 0, 0.0, v)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _run_linear(s):
    c = s["case"]
    if own:
        import moe_expert_ffn_router_amd as moe
        act = {"none": moe.ACT_NONE, "relu": moe.ACT_RELU, "silu": moe.ACT_SILU,
               "gelu": moe.ACT_GELU, "gelu_tanh": moe.ACT_GELU_TANH}[c["act"]]
        return [moe.linear(s["x"], s["w"], s["bias"], activation=act, gated=c["gated"],
                           residual=s["residual"], dtype=_DT[c["out_dtype"]])]
    v = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"]
    if c["gated"]:
        v = _act(c["act"], v[:, :c["N"]]) * v[:, c["N"]:]
    else:
        v = _act(c["act"], v)
    if s["residual"] is not None:
        v = s["residual"].float() + v
    return [v.to(_DT[c["out_dtype"]])]


_RUN = {"dispatch": _run_dispatch, "combine": _run_combine,
        "dispatch_backward": _run_dispatch_backward, "combine_backward": _run_combine_backward,
        "layer_norm": _run_layer_norm, "layer_norm_backward": _run_layer_norm_backward,
        "layer_norm_train": _run_layer_norm_train, "linear": _run_linear}


# ---------------------------------------------------------------- exact ---

def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    c, s = case, prepare(case, seed)
    d = {n: t.double() for n, t in s.items()
         if isinstance(t, torch.Tensor) and t.is_floating_point() and n != "rows"}
    if c["op"] == "linear":
        return _exact_linear(c, d)
    if c["op"].startswith("layer_norm"):
        return _exact_norm(c, s, d)
    # one slot of every token at a time, through the place of its expert in the lists
    T, k, H = c["T"], c["k"], c["H"]
    place = {}
    n = int(s["num_padded"])
    for p, slot in enumerate(s["sorted_ids"][:n].tolist()):
        if slot < T * k:
            place[slot] = p
    at = torch.tensor([place.get(i, -1) for i in range(T * k)], dtype=torch.int32).view(T, k)
    at = at.cuda()
    if c["op"] == "dispatch":
        rows = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for j in range(k):
            mine = at[:, j] >= 0
            rows[at[mine, j].long()] = d["x"][mine]
        return [rows, at]
    if c["op"] in ("combine", "dispatch_backward"):
        out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        for j in range(k):
            mine = at[:, j] >= 0
            term = s["rows"][at[mine, j].long()].double()
            out[mine] += term * d["weights"][mine, j, None] if c["op"] == "combine" else term
        return [out]
    drows = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    dweights = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        mine = at[:, j] >= 0
        where = at[mine, j].long()
        drows[where] = d["weights"][mine, j, None] * d["dout"][mine]
        dweights[mine, j] = torch.linalg.vecdot(d["dout"][mine], s["rows"][where].double())
    return [drows, dweights]


def _exact_norm(c, s, d):
    def centred(v):
        v = v - v.sum(1, keepdim=True) / c["H"]
        return v, 1 / (v.pow(2).sum(1, keepdim=True) / c["H"] + EPS).sqrt()

    result = []
    total = d.get("sum")
    if c["op"] != "layer_norm_backward":
        total = d["x"] * s["alpha"] + d.get("residual", 0)
        v, inv = centred(total)
        out = v * inv
        if c["affine"]:
            out = out * d["weight"] + d["bias"]
        result = [out, total] if c["residual"] or c["op"] == "layer_norm_train" else [out]
        if c["op"] == "layer_norm":
            return result
        # the backward pass takes the sum as the forward pass has stored it
        total = total.to(_DT[c["dtype"]]).double()
    v, inv = centred(total)
    g = d["dout"] * d["weight"] if c["affine"] else d["dout"]
    H = c["H"]
    ds = inv / H * (H * g - g.sum(1, keepdim=True)
                    - v * inv * inv * torch.linalg.vecdot(g, v).unsqueeze(1))
    if c["residual"]:
        ds = ds + d["dsum"]
    result.append(s["alpha"] * ds)
    if c["residual"]:
        result.append(ds)
    if c["affine"]:
        result.append(torch.linalg.vecdot(d["dout"].t(), (v * inv).t()))
    return result + [d["dout"].sum(0)]


def _exact_linear(c, d):
    def product(lo, hi):
        out = torch.matmul(d["w"][lo:hi], d["x"].t()).t()
        return out + d["bias"][lo:hi] if c["bias"] else out

    def act(v):
        if c["act"] == "relu":
            return v.clamp(min=0)
        if c["act"] == "silu":
            return v * torch.special.expit(v)
        if c["act"] == "gelu":
            return v * torch.special.ndtr(v)
        if c["act"] == "gelu_tanh":
            # (1 + tanh z) / 2 is the logistic function of 2 z
            return v * torch.special.expit(math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3))
        return v

    N = c["N"]
    out = act(product(0, N))
    if c["gated"]:
        out = out * product(N, 2 * N)
    return [out + d.get("residual", 0)]
