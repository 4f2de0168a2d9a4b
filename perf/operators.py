"""Measured cases of the operators around the expert FFN of an MoE layer: the
norms before and after it, the router projection in front of the routing, and
the low-rank adapters of many requests beside a projection they share.

``run`` computes a case in its plain form (elementary torch operations in fp32,
rounded once at the end) or, where ``own`` is set, through this library's entry
points. Sizes follow the library's workloads (hidden 4096 and 7168, 64 and 128
experts, top-8, batches of 16, 64 and 4096 tokens).
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-6


# ---------------------------------------------------------------- cases ---

def _norm_in(T, H, dtype="bf16", residual=True):
    return dict(op="norm_in", T=T, H=H, dtype=dtype, residual=residual)


def _norm_out(T, k, H, E, local, y_dtype="bf16", dtype="bf16", shared=False, post=False,
              residual=True, next=True):
    return dict(op="norm_out", T=T, k=k, H=H, E=E, local=local, y_dtype=y_dtype, dtype=dtype,
                shared=shared, post=post, residual=residual, next=next)


def _router(T, E, H, w_dtype="bf16", bias=False, dtype="bf16"):
    return dict(op="router", T=T, E=E, H=H, w_dtype=w_dtype, bias=bias, dtype=dtype)


def _lora(S, n, r, K, N, requests, x_dtype="bf16", y_dtype="bf16", aligned=True, skip=0.25):
    """S rows, n adapters of rank r; ``requests`` runs of consecutive rows that
    share an adapter (S: every row its own); ``aligned``: the row lists are in
    hand (one alignment serves every projection of a step) or made in the call;
    ``skip``: share of requests without an adapter."""
    return dict(op="lora", S=S, n=n, r=r, K=K, N=N, requests=requests, x_dtype=x_dtype,
                y_dtype=y_dtype, aligned=aligned, skip=skip)


def listed():
    return [
        # a decode step's residual add and norm in front of the router: latency
        dict(_norm_in(16, 4096), name="norm_in_decode_16x4096"),
        # the same for a prompt: one read and one write of two bf16 streams
        dict(_norm_in(4096, 4096), name="norm_in_prefill_4096x4096"),
        # the combine of a 16-token top-8 decode step with its residual and the next norm
        dict(_norm_out(16, 8, 4096, 64, 64), name="norm_out_decode_16x8x4096"),
        # 64 tokens of a W8A8 layer (fp32 expert outputs), gated shared expert, both norms
        dict(_norm_out(64, 8, 7168, 128, 128, y_dtype="f32", shared=True, post=True),
             name="norm_out_fp8_64x8x7168"),
        # a prompt, everything on: the largest case, bound by the experts' outputs
        dict(_norm_out(4096, 8, 4096, 128, 128, shared=True, post=True),
             name="norm_out_prefill_4096x8x4096"),
        # router projection of a decode step: latency
        dict(_router(16, 64, 4096), name="router_decode_16x64x4096"),
        # fp32 router weights, 64 tokens, a bias
        dict(_router(64, 128, 7168, w_dtype="f32", bias=True), name="router_f32w_64x128x7168"),
        # router projection of a prompt
        dict(_router(4096, 128, 4096), name="router_prefill_4096x128x4096"),
        # a decode step of 16 requests, each with an adapter of its own (or none), beside a
        # square projection
        dict(_lora(16, 16, 16, 4096, 4096, 16), name="lora_decode_16_r16_4096x4096"),
        # adapters of the experts' down projection: 64 tokens x top-8 slots over
        # 8 adapters x 128 experts, aligned in the call as a layer has to
        dict(_lora(512, 1024, 8, 2048, 7168, 512, aligned=False),
             name="lora_experts_512_r8_2048x7168"),
        # the same beside a W8A8 layer, whose intermediates are fp32
        dict(_lora(128, 1024, 16, 1536, 4096, 128, x_dtype="f32", y_dtype="f32", aligned=False),
             name="lora_experts_f32_128_r16_1536x4096"),
        # prompts of twelve requests over eight adapters of rank 64
        dict(_lora(4096, 8, 64, 4096, 4096, 12), name="lora_prefill_4096_r64_4096x4096"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult8(rng, lo, hi):
    return max(8, _log(rng, lo, hi) // 8 * 8)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("norm_in", "norm_out", "router", "lora"))
        if op == "norm_in":
            c = _norm_in(_log(rng, 1, 8192), _mult8(rng, 256, 8192),
                         rng.choice(("bf16", "bf16", "f32")), rng.random() < 0.8)
        elif op == "norm_out":
            E = rng.choice((8, 60, 64, 128, 160, 256))
            k = rng.choice((1, 2, 4, 6, 8))
            local = rng.choice((E, E, E // 4))
            c = _norm_out(_log(rng, 1, 4096), k, _mult8(rng, 256, 8192), E, local,
                          rng.choice(("bf16", "f32")), rng.choice(("bf16", "bf16", "f32")),
                          rng.random() < 0.5, rng.random() < 0.5,
                          local < E or rng.random() < 0.9, rng.random() < 0.7)
        elif op == "router":
            dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
            c = _router(_log(rng, 1, 4096), _log(rng, 4, 512), _mult8(rng, 256, 8192),
                        "f32" if dtype == "f32" else rng.choice(("bf16", "f32")),
                        rng.random() < 0.5, dtype)
        else:
            S = _log(rng, 1, 4096)
            n = _log(rng, 1, 64 if S > 1024 else 512)
            t = rng.choice(("bf16", "bf16", "bf16", "f32"))
            c = _lora(S, n, rng.choice((8, 16, 24, 32, 64, 128)), _mult8(rng, 256, 8192),
                      _mult8(rng, 256, 8192), S if S <= 256 else _log(rng, 1, 64), t, t,
                      rng.random() < 0.5, rng.choice((0.0, 0.25, 0.75)))
        if _cost(c) <= most:
            return c


def work(case):
    c = case
    if c["op"] == "norm_in":
        b = _BYTES[c["dtype"]]
        n = c["T"] * c["H"]
        streams = 2 + (2 if c["residual"] else 0)
        return {"bytes": n * b * streams + 4 * c["H"], "flops": 6 * n}
    if c["op"] == "norm_out":
        b, n = _BYTES[c["dtype"]], c["T"] * c["H"]
        slots = c["T"] * c["k"] * c["local"] / c["E"]
        streams = 1 + int(c["shared"]) + int(c["residual"]) + int(c["next"])
        byt = (slots * c["H"] * _BYTES[c["y_dtype"]] + n * b * streams + 8 * c["T"] * c["k"]
               + 4 * c["H"] * (int(c["post"]) + int(c["next"])) + 4 * c["T"] * int(c["shared"]))
        return {"bytes": byt, "flops": 2 * slots * c["H"] + 8 * n}
    if c["op"] == "router":
        T, E, H = c["T"], c["E"], c["H"]
        byt = T * H * _BYTES[c["dtype"]] + E * H * _BYTES[c["w_dtype"]] + 4 * T * E
        return {"bytes": byt + (4 * E if c["bias"] else 0), "flops": 2 * T * E * H}
    S, n, r, K, N = c["S"], c["n"], c["r"], c["K"], c["N"]
    live = S * (1 - c["skip"])
    seen = n * (1 - (1 - 1 / n) ** max(1, round(c["requests"] * (1 - c["skip"])))) if n > 1 else 1
    byt = (live * K * _BYTES[c["x_dtype"]] + 2 * live * N * _BYTES[c["y_dtype"]]
           + seen * r * (K + N) * 2 + 4 * S)
    return {"bytes": byt, "flops": 2 * live * r * (K + N)}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


# --------------------------------------------------------------- inputs ---

def _plan(ids, n, block_m):
    """Row lists of an alignment with block size block_m: (sorted_ids,
    block_adapter, num_padded), as a step keeps them for all its projections."""
    S = ids.numel()
    flat = ids.reshape(-1).long()
    cap = (S + min(n, S) * (block_m - 1) + block_m - 1) // block_m * block_m
    key = torch.where(flat < 0, n, flat)
    order = torch.argsort(key, stable=True)
    count = torch.bincount(key, minlength=n + 1)
    padded = (count[:n] + block_m - 1) // block_m * block_m
    ends = torch.cumsum(padded, 0)
    starts = ends - padded
    first = torch.cumsum(count, 0) - count
    k = key[order]
    live = k < n
    at = starts[k.clamp(max=n - 1)] + torch.arange(S, device=ids.device) - first[k]
    sid = torch.full((cap + 1,), S, dtype=torch.int32, device=ids.device)
    sid[torch.where(live, at, cap)] = torch.where(live, order, S).int()
    block = torch.arange(cap // block_m, device=ids.device) * block_m
    owner = torch.searchsorted(ends, block, right=True)
    adapter = torch.where(block < ends[-1], owner, -1).int()
    return sid[:cap].contiguous(), adapter, ends[-1:].int()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(1 + seed)

    def normal(*shape, dtype="f32", std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(_DT[dtype])

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    s = {"case": c}
    if c["op"] == "norm_in":
        # the hidden states a block adds to, and what the block before it gives
        s["x"] = normal(c["T"], c["H"], dtype=c["dtype"])
        s["residual"] = normal(c["T"], c["H"], dtype=c["dtype"], std=4.0) if c["residual"] else None
        s["weight"] = 1 + 0.1 * normal(c["H"])
        s["alpha"] = 0.75
    elif c["op"] == "norm_out":
        T, k, H, E = c["T"], c["k"], c["H"], c["E"]
        logits = normal(T, E)
        p, ids = torch.topk(torch.softmax(logits, 1), k, dim=1)
        # an expert-parallel rank holds the first `local` experts: the rows of
        # the other slots are never written, here NaN
        y = normal(T * k, H, dtype=c["y_dtype"])
        y[(ids >= c["local"]).reshape(-1)] = float("nan")
        s["y"], s["ids"], s["weights"] = y, ids.int().contiguous(), p.contiguous()
        s["shared"] = normal(T, H, dtype=c["dtype"]) if c["shared"] else None
        s["gate"] = normal(T) if c["shared"] else None
        s["residual"] = normal(T, H, dtype=c["dtype"], std=4.0) if c["residual"] else None
        s["weight"] = 1 + 0.1 * normal(H) if c["post"] else None
        s["next_weight"] = 1 + 0.1 * normal(H) if c["next"] else None
        s["scale"] = 0.5
    elif c["op"] == "router":
        s["x"] = normal(c["T"], c["H"], dtype=c["dtype"])
        s["w"] = normal(c["E"], c["H"], dtype=c["w_dtype"], std=c["H"] ** -0.5)
        s["bias"] = normal(c["E"], std=0.1) if c["bias"] else None
    else:
        S, n, r, K, N = c["S"], c["n"], c["r"], c["K"], c["N"]
        # runs of consecutive rows (a request each) share an adapter or have none (-1);
        # popular adapters first
        cuts = torch.randperm(S, generator=g, device="cuda")[:c["requests"]]
        request = torch.zeros(S, dtype=torch.long, device="cuda")
        request[cuts] = 1
        request = torch.cumsum(request, 0)
        adapter = (uniform(c["requests"] + 1) ** 1.5 * n).long().clamp(max=n - 1)
        adapter[uniform(c["requests"] + 1) < c["skip"]] = -1
        s["ids"] = adapter[request].int().reshape(S, 1)
        s["x"] = normal(S, K, dtype=c["x_dtype"])
        s["a"] = normal(n, r, K, dtype="bf16", std=K ** -0.5)
        s["b"] = normal(n, N, r, dtype="bf16", std=r ** -0.5)
        s["scale"] = 0.5 + uniform(n)
        s["y"] = normal(S, N, dtype=c["y_dtype"])
        s["out"] = s["y"].clone()  # rows without an adapter keep what the projection gave
        s["block_m"] = 64
        s["plan"] = _plan(s["ids"], n, 64) if c["aligned"] else None
    return s


# ------------------------------------------------------------------ run ---

def run(state):
    return _RUN[state["case"]["op"]](state)


def _rms(v, weight):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * weight


def _run_norm_in(s):
    if own:
        import moe_expert_ffn_router_amd as moe
        out, res = moe.norm_in(s["x"], s["weight"], residual=s["residual"], alpha=s["alpha"],
                               eps=EPS)
        return [out] if res is None else [out, res]
    v = s["alpha"] * s["x"].float()
    if s["residual"] is not None:
        v = s["residual"].float() + v
    out = _rms(v, s["weight"]).to(s["x"].dtype)
    return [out] if s["residual"] is None else [out, v.to(s["x"].dtype)]


def _run_norm_out(s):
    c = s["case"]
    dt = _DT[c["dtype"]]
    if own:
        import moe_expert_ffn_router_amd as moe
        out, nxt = moe.norm_out(s["y"], s["weights"], topk_ids=s["ids"], num_experts=c["local"],
                                shared=s["shared"], gate=s["gate"], residual=s["residual"],
                                weight=s["weight"], next_weight=s["next_weight"],
                                scale=s["scale"], eps=EPS, dtype=dt)
        return [out] if nxt is None else [out, nxt]
    here = (s["ids"] < c["local"]).unsqueeze(-1)
    y = torch.where(here, s["y"].view(c["T"], c["k"], c["H"]).float(), 0.0)
    v = (y * s["weights"].unsqueeze(-1)).sum(1)
    if s["shared"] is not None:
        v = v + torch.sigmoid(s["gate"]).unsqueeze(-1) * s["shared"].float()
    if s["weight"] is not None:
        v = _rms(v, s["weight"])
    v = s["scale"] * v
    if s["residual"] is not None:
        v = s["residual"].float() + v
    if s["next_weight"] is None:
        return [v.to(dt)]
    return [v.to(dt), _rms(v, s["next_weight"]).to(dt)]


def _run_router(s):
    if own:
        import moe_expert_ffn_router_amd as moe
        return [moe.router_logits(s["x"], s["w"], bias=s["bias"])]
    logits = s["x"].float() @ s["w"].float().t()
    return [logits if s["bias"] is None else logits + s["bias"]]


def _run_lora(s):
    c = s["case"]
    n, r = c["n"], c["r"]
    if own:
        import moe_expert_ffn_router_amd as moe
        plan = s["plan"]
        if plan is None:
            plan = moe.align_block(s["ids"], n, s["block_m"])
        return [moe.lora_add(s["y"], s["x"], s["a"], s["b"], *plan, s["block_m"],
                             scale=s["scale"], out=s["out"])]
    ids = s["ids"].reshape(-1).long()
    has, at = ids >= 0, ids.clamp(min=0)
    x = s["x"].float()
    # each row's own factors, or all adapters' products and a choice among them: whichever
    # costs less
    if c["S"] <= n or n >= 128:
        z = torch.bmm(s["a"][at].float(), x.unsqueeze(-1))
        d = torch.bmm(s["b"][at].float(), z).squeeze(-1)
    else:
        z = (x @ s["a"].reshape(n * r, -1).float().t()).view(-1, n, r)
        z = torch.where((torch.arange(n, device=ids.device) == at[:, None]).unsqueeze(-1), z, 0.0)
        d = z.reshape(-1, n * r) @ s["b"].float().transpose(1, 2).reshape(n * r, -1)
    d = d * torch.where(has, s["scale"][at], 0.0).unsqueeze(-1)
    return [(s["y"].float() + d).to(s["y"].dtype)]


_RUN = {"norm_in": _run_norm_in, "norm_out": _run_norm_out, "router": _run_router,
        "lora": _run_lora}


# ---------------------------------------------------------------- exact ---

def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}

    def unit(rows):  # divide each row by its root mean square
        return rows / (rows.pow(2).sum(1, keepdim=True) / rows.shape[1] + EPS).sqrt()

    op = case["op"]
    if op == "norm_in":
        total = d["x"] * s["alpha"] + d.get("residual", 0)
        out = unit(total) * d["weight"]
        return [out, total] if case["residual"] else [out]
    if op == "norm_out":
        T, k, H = case["T"], case["k"], case["H"]
        rows = d["y"].view(T, k, H)
        total = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(k):
            mine = s["ids"][:, j] < case["local"]
            total[mine] += rows[mine, j] * d["weights"][mine, j, None]
        if case["shared"]:
            total += d["shared"] / (1 + torch.exp(-d["gate"]))[:, None]
        if case["post"]:
            total = unit(total) * d["weight"]
        total = total * s["scale"] + d.get("residual", 0)
        return [total, unit(total) * d["next_weight"]] if case["next"] else [total]
    if op == "router":
        out = torch.matmul(d["w"], d["x"].t()).t()
        return [out + d["bias"] if case["bias"] else out]
    out = d["y"].clone()
    ids = s["ids"].view(-1)
    for a in sorted(set(ids.tolist()) - {-1}):
        rows = (ids == a).nonzero().view(-1)
        z = torch.matmul(d["x"][rows], d["a"][a].t())
        out[rows] += d["scale"][a] * torch.matmul(z, d["b"][a].t())
    return [out]
