"""The operators around the routed experts, each with its plain form.

Three families, as one layer of a mixture-of-experts decoder calls them in turn:

* ``norm``: the residual join behind a block (second branch and its gate, post
  norm, gate, residual scale) fused with the norm before the next block;
* ``route``: scored routing (softmax or sigmoid scores, a selection bias,
  expert groups, top-k, renormalised and scaled weights) with the optional
  lists of each expert's pairs;
* ``q8``: a dense product in 8-bit integers, activations quantised per token
  on the fly, weights held as int8 with one scale per output channel.

A case is a dict of sizes, types and switches.  ``run`` computes it with
elementary torch operations, or through ``expert_offload_b200`` where ``own``
is true; ``exact`` computes it in 64 bits from the definition.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# --------------------------------------------------------------------- cases

def _route(name, T, E, k, score, groups, topk_groups, group_top, bias, renorm, scale, dtype, lists):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "groups": groups,
            "topk_groups": topk_groups, "group_top": group_top, "bias": bias, "renorm": renorm,
            "scale": scale, "dtype": dtype, "lists": lists}


def _norm(name, T, H, x, y, shared, post, gate, next_, alpha, beta, offset):
    return {"name": name, "op": "norm", "T": T, "H": H, "x": x, "y": y, "shared": shared, "post": post,
            "gate": gate, "next": next_, "alpha": alpha, "beta": beta, "offset": offset}


def _q8(name, T, K, N, x, y):
    return {"name": name, "op": "q8", "T": T, "K": K, "N": N, "x": x, "y": y}


def listed():
    return [
        # one decoded token of the 256-expert layer, sigmoid scores balanced by a bias, 4 of 8 groups
        _route("route_token", 1, 256, 8, "sigmoid", 8, 4, 2, True, True, 2.5, "f32", False),
        # a verify batch over 512 experts, plain softmax with a balance bias
        _route("route_verify", 8, 512, 8, "softmax", 1, 1, 1, True, True, 1.0, "f32", False),
        # a ragged chunk: bf16 logits, 3 of 8 groups of 20 experts by their best member, weights not renormalised
        _route("route_ragged", 1237, 160, 6, "softmax", 8, 3, 1, False, False, 16.0, "bf16", True),
        # the largest prefill chunk, with the lists that the batched experts read
        _route("route_prefill", 8192, 512, 8, "sigmoid", 8, 4, 2, True, True, 2.5, "f32", True),
        # one decoded token: routed and shared branch joined, post norm, then the next block's norm
        _norm("norm_token", 1, 2048, "bf16", "f32", True, True, "none", True, 1.0, 1.0, 0.0),
        # odd row length, f32 stream, per-channel gate, scaled residual
        _norm("norm_ragged", 333, 1001, "f32", "f32", False, True, "channel", True, 0.5, 0.25, 1.0),
        # the largest prefill chunk of the 2048-wide layer
        _norm("norm_prefill", 8192, 2048, "bf16", "f32", True, True, "token", True, 1.0, 1.0, 0.0),
        # the widest rows, a gate for each element
        _norm("norm_wide", 2048, 8192, "bf16", "bf16", False, True, "full", True, 1.0, 0.5, 0.0),
        # one decoded token through the gate and up rows of a 512-wide shared expert
        _q8("q8_token", 1, 2048, 1024, "bf16", "bf16"),
        # a verify batch through a wide dense product
        _q8("q8_verify", 5, 2048, 8192, "bf16", "f32"),
        # odd everything
        _q8("q8_ragged", 517, 2001, 1503, "f32", "f32"),
        # the largest prefill chunk through the largest square product
        _q8("q8_prefill", 8192, 8192, 8192, "bf16", "bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm uniform."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "norm", "q8"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _spread(rng, 8, 512 // groups)
        E = groups * size
        topk_groups = rng.randint((groups + 1) // 2, groups)
        k = rng.randint(1, min(16, topk_groups * size))
        T = _spread(rng, 1, 8192)
        return {"op": "route", "T": T, "E": E, "k": k, "score": rng.choice(["softmax", "sigmoid"]),
                "groups": groups, "topk_groups": topk_groups, "group_top": rng.choice([1, 2]),
                "bias": rng.random() < 0.6, "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5, 16.0]),
                "dtype": rng.choice(["f32", "bf16"]), "lists": rng.random() < 0.5}
    if op == "norm":
        H = _spread(rng, 64, 8192)
        if rng.random() < 0.6:
            H = max(64, H // 64 * 64)
        T = _spread(rng, 1, min(8192, max(1, (1 << 24) // H)))
        return {"op": "norm", "T": T, "H": H, "x": rng.choice(["f32", "bf16"]), "y": rng.choice(["f32", "bf16"]),
                "shared": rng.random() < 0.5, "post": rng.random() < 0.7,
                "gate": rng.choice(["none", "token", "channel", "full"]), "next": rng.random() < 0.8,
                "alpha": rng.choice([1.0, 0.5]), "beta": rng.choice([1.0, 0.25]), "offset": rng.choice([0.0, 1.0])}
    K, N = _spread(rng, 128, 8192), _spread(rng, 128, 8192)
    if rng.random() < 0.6:
        K, N = K // 64 * 64, N // 64 * 64
    return {"op": "q8", "T": _spread(rng, 1, 8192), "K": K, "N": N, "x": rng.choice(["f32", "bf16"]),
            "y": rng.choice(["f32", "bf16"])}


# -------------------------------------------------------------------- inputs

def _up16(n):
    return -(-n // 16) * 16


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype="f32", std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(_DT[dtype])

    def empty(*shape, dtype):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    s = dict(case)
    T = case["T"]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        s["logits"] = randn(T, E, dtype=case["dtype"])
        # a balance bias is of the scores' own size
        s["sel_bias"] = randn(E, std=0.1 if case["score"] == "sigmoid" else 0.5 / E) if case["bias"] else None
        s["idx"], s["wts"] = empty(T, k, dtype=torch.int32), empty(T, k, dtype=torch.float32)
        if case["lists"]:
            s["cnt"], s["off"], s["perm"] = (empty(n, dtype=torch.int32) for n in (E, E + 1, T * k))
        if own:
            import expert_offload_b200 as eo
            s["rule"] = eo.RouteRule(score=eo.SCORE_SIGMOID if case["score"] == "sigmoid" else eo.SCORE_SOFTMAX,
                                     n_groups=case["groups"], topk_groups=case["topk_groups"],
                                     group_top=case["group_top"], renormalise=case["renorm"], scale=case["scale"])
            n = eo.moe_route_scored_workspace_bytes(T, E, k)
            s["ws"] = torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda") if case["lists"] else None
    elif case["op"] == "norm":
        H = case["H"]
        s["xv"] = randn(T, H, dtype=case["x"])
        s["yv"] = randn(T, H, dtype=case["y"], std=0.3)
        s["y2"] = randn(T, H, dtype=case["y"], std=0.3) if case["shared"] else None
        s["y2_gate"] = randn(T) if case["shared"] else None
        c = 1.0 - case["offset"]
        s["w_post"] = (randn(H, std=0.1) + c).to(_DT[case["x"]]) if case["post"] else None
        s["w_pre"] = (randn(H, std=0.1) + c).to(_DT[case["x"]]) if case["next"] else None
        shape = {"none": None, "token": (T,), "channel": (H,), "full": (T, H)}[case["gate"]]
        s["gv"] = randn(*shape) if shape else None
        s["x_out"] = torch.empty_like(s["xv"])
        s["xn"] = torch.empty_like(s["xv"]) if case["next"] else None
        if own:
            import expert_offload_b200 as eo
            kind = {"none": eo.GATE_NONE, "token": eo.GATE_TOKEN, "channel": eo.GATE_CHANNEL,
                    "full": eo.GATE_FULL}[case["gate"]]
            s["rule"] = eo.NormRule(w_post=s["w_post"], w_pre=s["w_pre"], w_dtype=_own_dtype(eo, case["x"]),
                                    eps=1e-6, w_offset=case["offset"], residual_scale=case["alpha"],
                                    branch_scale=case["beta"], gate_kind=kind, gate_act=eo.GATE_SIGMOID)
    else:
        K, N = case["K"], case["N"]
        s["xv"] = randn(T, K, dtype=case["x"])
        # the weights as a program holds them: int8 rows padded to whole 16-byte units, one scale per row
        w = randn(N, K, std=0.02)
        top = w.abs().amax(1)
        s["wq"] = torch.zeros(N, _up16(K), dtype=torch.int8, device="cuda")
        s["wq"][:, :K] = torch.round(w * (127.0 / top)[:, None]).clamp_(-127, 127).to(torch.int8)
        s["w_scale"] = top / 127.0
        s["out"] = empty(T, N, dtype=_DT[case["y"]])
        if own:
            import expert_offload_b200 as eo
            s["ws"] = torch.zeros(eo.q8_linear_workspace_bytes(T, K, N), dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------------- the calls

def _own_dtype(eo, name):
    return eo.HFQ_F32 if name == "f32" else eo.HFQ_BF16


def _run_own(s):
    import expert_offload_b200 as eo
    if s["op"] == "route":
        lists = {n: s[n] for n in ("cnt", "off", "perm")} if s["lists"] else {}
        eo.moe_route_scored(s["logits"], _own_dtype(eo, s["dtype"]), s["T"], s["E"], s["k"], s["rule"],
                            s["idx"], s["wts"], bias=s["sel_bias"], workspace=s["ws"], **lists)
        return {"idx": s["idx"], "wts": s["wts"], **lists}
    if s["op"] == "norm":
        dt = _own_dtype(eo, s["x"])
        eo.moe_norm_residual(s["rule"], s["T"], s["H"], s["xv"], dt, y=s["yv"], y_dtype=_own_dtype(eo, s["y"]),
                             y2=s["y2"], y2_gate=s["y2_gate"], gate=s["gv"], x_out=s["x_out"], xn=s["xn"],
                             xn_dtype=dt)
        return {"x": s["x_out"], "xn": s["xn"]}
    eo.q8_linear(s["xv"], _own_dtype(eo, s["x"]), s["T"], s["K"], s["wq"], s["w_scale"], s["N"], s["out"],
                 _own_dtype(eo, s["y"]), s["ws"], ldw=s["wq"].shape[1])
    return {"y": s["out"]}


# --------------------------------------------------------------- plain forms

def _plain_route(s):
    # selection compares sums of scores and biases that can lie next to each other: 64 bits
    T, E, k = s["T"], s["E"], s["k"]
    l = s["logits"].double()
    if s["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        score = torch.exp(l - l.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    c = score if s["sel_bias"] is None else score + s["sel_bias"].double()
    if s["groups"] > 1:
        by = c.view(T, s["groups"], E // s["groups"])
        best = torch.sort(by, dim=2, descending=True).values[:, :, :s["group_top"]].sum(2)
        at = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        keep = torch.zeros(T, s["groups"], dtype=torch.bool, device=l.device).scatter_(1, at, True)
        c = torch.where(keep[:, :, None], by, -math.inf).reshape(T, E)
    idx = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(score, 1, idx)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    out = {"idx": idx.to(torch.int32), "wts": (w * s["scale"]).float()}
    if s["lists"]:
        flat = idx.reshape(-1)
        cnt = torch.zeros(E, dtype=torch.int64, device=l.device).scatter_add_(0, flat, torch.ones_like(flat))
        off = torch.zeros(E + 1, dtype=torch.int64, device=l.device)
        off[1:] = torch.cumsum(cnt, 0)
        perm = torch.sort(flat, stable=True).indices
        out.update(cnt=cnt.to(torch.int32), off=off.to(torch.int32), perm=perm.to(torch.int32))
    return out


def _rms(v, w, offset):
    return v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * (w.to(v.dtype) + offset)


def _join(s, f):
    """The new residual stream in type f, not yet rounded."""
    b = s["yv"].to(f)
    if s["y2"] is not None:
        b = b + torch.sigmoid(s["y2_gate"].to(f))[:, None] * s["y2"].to(f)
    if s["post"]:
        b = _rms(b, s["w_post"], s["offset"])
    if s["gv"] is not None:
        gate = torch.sigmoid(s["gv"].to(f))
        b = b * (gate[:, None] if s["gate"] == "token" else gate)
    return s["alpha"] * s["xv"].to(f) + s["beta"] * b


def _plain_norm(s):
    x = _join(s, torch.float32).to(_DT[s["x"]])
    xn = _rms(x.float(), s["w_pre"], s["offset"]).to(_DT[s["x"]]) if s["next"] else None
    return {"x": x, "xn": xn}


def _quantised(x):
    """int8 values (held in f64) and their scales: q = x * 127 / max|x| to the nearest, ties to even."""
    x = x.double()  # quotients lie next to rounding borders
    top = x.abs().amax(1, keepdim=True)
    q = torch.where(top > 0, torch.round(x * 127.0 / top), 0.0)
    return q, top / 127.0


def _plain_q8(s):
    q, scale = _quantised(s["xv"])
    acc = q.float() @ s["wq"][:, :s["K"]].float().t()
    return {"y": (acc * scale.float() * s["w_scale"]).to(_DT[s["y"]])}


def run(state):
    if own:
        return _run_own(state)
    return {"route": _plain_route, "norm": _plain_norm, "q8": _plain_q8}[state["op"]](state)


# -------------------------------------------------------------- 64-bit truth

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        # whole numbers are compared as such; the weights follow from the plain form's selection rule,
        # found here by ranking each expert against all others
        T, E, k = case["T"], case["E"], case["k"]
        step = max(1, (1 << 26) // (E * E))
        weights = []
        for t0 in range(0, T, step):
            l = s["logits"][t0:t0 + step].double()
            p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
            c = p + (s["sel_bias"].double() if case["bias"] else 0.0)
            n = case["groups"]
            top = torch.topk(c.view(-1, n, E // n), case["group_top"], dim=2).values.sum(2)
            order = torch.arange(n, device=l.device)
            ahead = (top[:, None, :] > top[:, :, None]) | ((top[:, None, :] == top[:, :, None]) & (order[None, :] < order[:, None]))
            live = (ahead.sum(2) < case["topk_groups"]).repeat_interleave(E // n, dim=1)
            c = torch.where(live, c, -math.inf)
            order = torch.arange(E, device=l.device)
            ahead = (c[:, None, :] > c[:, :, None]) | ((c[:, None, :] == c[:, :, None]) & (order[None, :] < order[:, None]))
            rank = ahead.sum(2)
            w = torch.zeros(l.shape[0], E, dtype=torch.float64, device=l.device).scatter_(1, rank, p)[:, :k]
            if case["renorm"]:
                w = w / w.sum(1, keepdim=True)
            weights.append(w * case["scale"])
        return {"idx": None, "wts": torch.cat(weights), **({"cnt": None, "off": None, "perm": None} if case["lists"] else {})}
    if case["op"] == "norm":
        x = _exact_join(s)
        # the stream is rounded to its type before it is normed again
        r = x.to(_DT[case["x"]]).double()
        xn = r / (r.square().mean(1, keepdim=True) + 1e-6).sqrt() * (s["w_pre"].double() + case["offset"]) if case["next"] else None
        return {"x": x, "xn": xn}
    x = s["xv"].double()
    top = x.abs().amax(1, keepdim=True)
    q = (x * 127.0 / top).round()
    acc = q @ s["wq"][:, :case["K"]].double().t()
    return {"y": acc * (top / 127.0) * s["w_scale"].double()}


def _exact_join(s):
    b = s["yv"].double()
    if s["shared"]:
        b = b + s["y2"].double() / (1.0 + torch.exp(-s["y2_gate"].double()))[:, None]
    if s["post"]:
        b = b / (b.square().mean(1, keepdim=True) + 1e-6).sqrt() * (s["w_post"].double() + s["offset"])
    if s["gate"] != "none":
        d = 1.0 + torch.exp(-s["gv"].double())
        b = b / (d[:, None] if s["gate"] == "token" else d)
    return s["alpha"] * s["xv"].double() + s["beta"] * b


# ---------------------------------------------------------------------- work

_SIZE = {"f32": 4, "bf16": 2}


def work(case):
    T = case["T"]
    if case["op"] == "route":
        E, k = case["E"], case["k"]
        b = T * E * _SIZE[case["dtype"]] + 8 * T * k + (4 * E if case["bias"] else 0)
        if case["lists"]:
            b += 4 * (T * k + 2 * E + 1)
        return {"bytes": b, "flops": 4 * T * E}
    if case["op"] == "norm":
        H, sx, sy = case["H"], _SIZE[case["x"]], _SIZE[case["y"]]
        b = T * H * (sx * (3 if case["next"] else 2) + sy * (2 if case["shared"] else 1))
        b += {"none": 0, "token": 4 * T, "channel": 4 * H, "full": 4 * T * H}[case["gate"]]
        b += H * sx * (int(case["post"]) + int(case["next"])) + (4 * T if case["shared"] else 0)
        return {"bytes": b, "flops": 10 * T * H}
    K, N = case["K"], case["N"]
    return {"bytes": T * K * _SIZE[case["x"]] + N * K + 4 * N + T * N * _SIZE[case["y"]], "flops": 2 * T * K * N}
