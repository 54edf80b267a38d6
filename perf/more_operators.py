"""The rest of a pre-norm MLP or mixture-of-experts block: the cases that are timed, and their plain forms.

Operators, each reached through the package's public entry points:

- route: a router's choice from its logits: softmax or sigmoid scores, a bias that only the choice sees,
  groups of experts, top-k, renormalised weights (``gf_route_execute``, backward ``gf_route_grad_execute``).
- norm: root-mean-square norm with the residual's addition before it, 16-bit or e4m3 output with a scale for
  each block of 128 (``gf_rmsnorm_execute``, backward ``gf_rmsnorm_grad_execute``).
- residual: out = act(A B + bias) + residual in one kernel (``gf_matmul_residual_execute``); backward, the
  gradient of what the activation took and of the bias (``gf_dact_bgrad_execute``).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token of a serving loop over grouped experts with a balancing bias: nothing but latency
        dict(name="route-token", op="route", direction="forward", tokens=1, experts=256, topk=8, groups=8, topk_groups=4, best=2,
             score="sigmoid", bias=True, renorm=True, scale=2.5, dtype="fp32", masked=0.0),
        # a training step's micro-batch over the same kind of router
        dict(name="route-train", op="route", direction="forward", tokens=16384, experts=256, topk=8, groups=8, topk_groups=4, best=2,
             score="sigmoid", bias=True, renorm=True, scale=2.5, dtype="fp32", masked=0.0),
        # its gradient for the softmax router, on 16-bit logits
        dict(name="route-grad", op="route", direction="backward", tokens=16384, experts=128, topk=8, groups=1, topk_groups=1, best=1,
             score="softmax", bias=False, renorm=True, scale=1.0, dtype="bf16", masked=0.0),
        # one token of a serving loop before an 8-bit product
        dict(name="norm-token", op="norm", direction="fp8", rows=1, hidden=5120, residual=True, dtype="bf16"),
        # a prompt before an 8-bit product
        dict(name="norm-fp8-prompt", op="norm", direction="fp8", rows=16384, hidden=5120, residual=True, dtype="bf16"),
        # a width that no vector load divides
        dict(name="norm-odd", op="norm", direction="forward", rows=5003, hidden=2047, residual=True, dtype="fp16"),
        # a training step's gradient, with the one that comes along the residual
        dict(name="norm-grad-train", op="norm", direction="backward", rows=16384, hidden=4096, residual=True, dtype="bf16"),
        # one token through the MLP's down projection: the weight is read once
        dict(name="residual-token", op="residual", direction="forward", m=1, n=5120, k=17408, act="none", bias=False, save=False, layout="nk", dtype="bf16"),
        # a batch of single tokens, the weight stored the other way, with a bias
        dict(name="residual-decode", op="residual", direction="forward", m=48, n=4096, k=16384, act="none", bias=True, save=False, layout="kn", dtype="fp16"),
        # a prompt through the down projection
        dict(name="residual-prompt", op="residual", direction="forward", m=8192, n=5120, k=17408, act="none", bias=False, save=False, layout="nk", dtype="bf16"),
        # a residual MLP layer of odd sizes in training: GELU, its argument saved
        dict(name="residual-odd", op="residual", direction="forward", m=1003, n=2056, k=1000, act="gelu", bias=True, save=True, layout="kn", dtype="fp16"),
        # that layer's gradient at a training step's size
        dict(name="residual-grad", op="residual", direction="backward", m=8192, n=16384, k=0, act="gelu", bias=True, save=True, layout="nk", dtype="bf16"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    while True:
        case = _draw(rng)
        w, most = work(case), {"bytes": 0.0, "flops": 0.0}
        for c in listed():
            if c["op"] == case["op"]:
                most = {k: max(most[k], work(c)[k]) for k in most}
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return case


def _draw(rng):
    op = rng.choice(("route", "norm", "residual"))
    if op == "route":
        size = rng.choice((1, 2, 3, 4, 5, 8, 16, 32, 60, 64, 128))  # of a group
        groups = rng.choice((1, 1, 2, 3, 4, 8, 16))
        experts = max(2, size * groups)
        groups = groups if size * groups == experts else 1
        keep = rng.randint(1, groups)
        score = rng.choice(("softmax", "sigmoid"))
        return dict(op=op, direction=rng.choice(("forward", "forward", "backward")), tokens=_log(rng, 1, 16384), experts=experts,
                    topk=rng.randint(1, min(10, experts // groups * keep)), groups=groups, topk_groups=keep, best=rng.choice((1, 2)),
                    score=score, bias=rng.choice((True, False)), renorm=rng.choice((True, False)), scale=rng.choice((1.0, 2.5)),
                    dtype=rng.choice(("fp32", "bf16", "fp16")), masked=rng.choice((0.0, 0.0, 0.1)))
    dtype = rng.choice(("bf16", "fp16"))
    if op == "norm":
        direction = rng.choice(("forward", "backward", "fp8"))
        hidden = 16 * _log(rng, 4, 1024)
        if direction != "fp8":
            hidden += rng.choice((0, 0, 0, 1, 6, 8))
        return dict(op=op, direction=direction, rows=_log(rng, 1, 16384), hidden=hidden, residual=rng.choice((True, True, False)), dtype=dtype)
    backward = rng.random() < 0.25
    return dict(op=op, direction="backward" if backward else "forward", m=_log(rng, 1, 8192), n=8 * _log(rng, 8, 2048),
                k=0 if backward else 8 * _log(rng, 8, 2176), act=rng.choice(("none", "relu", "gelu", "silu")), bias=rng.choice((True, False)),
                save=rng.choice((True, False)), layout=rng.choice(("nk", "kn")), dtype=dtype)


def _ceil(a, b):
    return -(-a // b)


def work(case):
    """Each input read once, each output written once; one pass of arithmetic."""
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        logits = t * e * (4 if case["dtype"] == "fp32" else 2)
        if case["direction"] == "forward":
            return {"bytes": logits + e * 4 * case["bias"] + 8 * t * k, "flops": 4 * t * e}
        return {"bytes": 2 * logits + 8 * t * k, "flops": 6 * t * e}
    if case["op"] == "norm":
        m, h, extra = case["rows"], case["hidden"], int(case["residual"])
        if case["direction"] == "backward":
            return {"bytes": 2 * m * h * (3 + extra) + 6 * h, "flops": 11 * m * h}
        out = m * h + 4 * m * _ceil(h, 128) if case["direction"] == "fp8" else 2 * m * h
        return {"bytes": 2 * m * h * (1 + 2 * extra) + 2 * h + out, "flops": 6 * m * h}
    m, n, k = case["m"], case["n"], case["k"]
    if case["direction"] == "backward":
        plain = case["act"] == "none"
        return {"bytes": 2 * m * n * (1 if plain else 3) + 4 * n, "flops": m * n * (1 if plain else 10)}
    return {"bytes": 2 * (m * k + n * k + m * n * (2 + case["save"]) + n * case["bias"]), "flops": 2 * m * n * k}


# ---------------------------------------------------------------- the inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activations(gen, rows, cols, dtype):
    """Hidden states: rows of different size, a few channels much larger than the rest."""
    x = _randn(gen, rows, cols) * torch.exp(0.5 * _randn(gen, rows, 1)) * torch.exp(0.5 * _randn(gen, 1, cols))
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    state = {"case": case}
    if op == "route":
        t, e = case["tokens"], case["experts"]
        logits = (_randn(gen, t, e) + 0.3 * _randn(gen, e)).to(dtype)
        if case["masked"]:  # experts that are switched off
            logits[:, torch.rand(e, generator=gen, device="cuda") < case["masked"]] = -math.inf
        state["logits"] = logits
        size = 0.05 if case["score"] == "sigmoid" else 0.2 / e
        state["bias"] = size * _randn(gen, e) if case["bias"] else None
        if case["direction"] == "backward":
            state["expert"] = _choose(case, state)
            state["d_weight"] = _randn(gen, t, case["topk"])
    elif op == "norm":
        m, h = case["rows"], case["hidden"]
        state["x"] = _activations(gen, m, h, dtype)
        state["weight"] = (1 + 0.2 * _randn(gen, h)).to(dtype)
        state["residual"] = _activations(gen, m, h, dtype) if case["residual"] else None
        if case["direction"] == "backward":
            state["d_out"] = _randn(gen, m, h).to(dtype)
    else:
        m, n, k = case["m"], case["n"], case["k"]
        state["bias"] = (0.1 * _randn(gen, n)).to(dtype) if case["bias"] else None
        if case["direction"] == "forward":
            state["a"] = _activations(gen, m, k, dtype)
            shape = (n, k) if case["layout"] == "nk" else (k, n)
            state["b"] = (_randn(gen, *shape) / math.sqrt(k)).to(dtype)
            state["residual"] = _activations(gen, m, n, dtype)
        else:
            state["z"] = _randn(gen, m, n).to(dtype) if case["act"] != "none" else None
            state["d_out"] = _randn(gen, m, n).to(dtype)
    if own:
        _plan(state)
    return state


def _plan(state):
    """The plans and the output buffers that a program keeps from step to step."""
    import gemm_epilogue_tmem_gb300 as gf

    case, op = state["case"], state["case"]["op"]
    dtype = DTYPES[case["dtype"]]
    code = {"fp16": gf.GF_F16, "bf16": gf.GF_BF16, "fp32": gf.GF_F32}[case["dtype"]]

    def new(*shape, dtype=dtype):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        score = gf.GF_SCORE_SOFTMAX if case["score"] == "softmax" else gf.GF_SCORE_SIGMOID
        state["plan"] = gf.gf_route_plan(t, e, k, code, score, renorm=case["renorm"], scale=case["scale"], groups=case["groups"],
                                         topk_groups=case["topk_groups"], group_best=case["best"])
        if case["direction"] == "forward":
            out = {"expert": new(t, k, dtype=torch.int32), "weight": new(t, k, dtype=torch.float32)}
        else:
            out = {"d_logits": new(t, e)}
    elif op == "norm":
        m, h = case["rows"], case["hidden"]
        state["plan"] = gf.gf_rmsnorm_plan(m, h, code, EPS)
        if case["direction"] == "backward":
            out = {"d_x": new(m, h), "d_weight": new(h, dtype=torch.float32)}
        elif case["direction"] == "fp8":
            out = {"q": new(m, h, dtype=torch.float8_e4m3fn), "scale": new(m, _ceil(h, 128), dtype=torch.float32)}
        else:
            out = {"out": new(m, h)}
        if case["residual"] and case["direction"] != "backward":
            out["residual"] = new(m, h)
    else:
        m, n = case["m"], case["n"]
        act = {"none": gf.GF_ACT_NONE, "relu": gf.GF_ACT_RELU, "gelu": gf.GF_ACT_GELU, "silu": gf.GF_ACT_SILU}[case["act"]]
        if case["direction"] == "forward":
            layout = gf.GF_B_NK if case["layout"] == "nk" else gf.GF_B_KN
            state["plan"] = gf.gf_matmul_residual_plan(m, n, case["k"], code, act, layout)
            out = {"out": new(m, n)}
            if case["save"]:
                out["z"] = new(m, n)
        else:
            state["plan"] = gf.gf_dact_bgrad_plan(m, n, code, act)
            out = {"bgrad": new(n, dtype=torch.float32)}
            if case["act"] != "none":
                out["d_z"] = new(m, n)
    state["out"] = out


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import gemm_epilogue_tmem_gb300 as gf

    case, out = state["case"], state["out"]
    op, direction = case["op"], case["direction"]
    if op == "route" and direction == "forward":
        gf.gf_route_execute(state["plan"], state["logits"], out["expert"], out["weight"], bias=state["bias"])
    elif op == "route":
        gf.gf_route_grad_execute(state["plan"], state["logits"], state["expert"], state["d_weight"], out["d_logits"])
    elif op == "norm" and direction == "backward":
        gf.gf_rmsnorm_grad_execute(state["plan"], state["d_out"], state["x"], state["weight"], out["d_x"], d_weight=out["d_weight"],
                                   d_residual=state["residual"])
    elif op == "norm":
        gf.gf_rmsnorm_execute(state["plan"], state["x"], state["weight"], residual=state["residual"], residual_out=out.get("residual"),
                              out=out.get("out"), out8=out.get("q"), out_scale=out.get("scale"))
    elif direction == "forward":
        gf.gf_matmul_residual_execute(state["plan"], state["a"], state["b"], state["residual"], out["out"], bias=state["bias"],
                                      z_out=out.get("z"))
    else:
        gf.gf_dact_bgrad_execute(state["plan"], state["d_out"], z=state["z"], d_z=out.get("d_z"), bgrad=out["bgrad"])
    return out


# ---------------------------------------------------------------- the plain forms
def _scores(case, logits):
    if case["score"] == "softmax":
        top = logits.amax(1, keepdim=True)
        e = torch.exp(logits - torch.where(torch.isinf(top), 0.0, top))
        return e / e.sum(1, keepdim=True).clamp(min=1e-300 if e.dtype == torch.float64 else 1e-30)
    e = torch.exp(-logits.abs())
    return torch.where(logits >= 0, 1.0, e) / (1 + e)


def _choose(case, state):
    """The chosen experts, best first, ties to the lowest index; -1 where a mask leaves fewer than topk. Ranked in 64
    bits: whole numbers depend on scores that lie next to each other."""
    logits = state["logits"].double()
    t, e, g = case["tokens"], case["experts"], case["groups"]
    off = torch.isneginf(logits)
    ranked = logits  # without a bias the scores are in the logits' order
    score = _scores(case, logits)
    if state["bias"] is not None:
        ranked = torch.where(off, -math.inf, score + state["bias"].double())
    if g > 1:
        of_groups = ranked
        if case["best"] == 2 and state["bias"] is None:
            of_groups = torch.where(off, -math.inf, score)  # sums are of scores
        best = torch.sort(of_groups.view(t, g, e // g), dim=2, descending=True).values[:, :, :min(case["best"], e // g)]
        total = torch.where(torch.isneginf(best), 0.0, best).sum(2)
        total = torch.where(torch.isneginf(best[:, :, 0]), -math.inf, total)
        order = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        stays = torch.zeros(t, g, dtype=torch.bool, device=logits.device).scatter_(1, order, True)
        ranked = torch.where(stays.repeat_interleave(e // g, 1), ranked, -math.inf)
    value, expert = torch.sort(ranked, dim=1, descending=True, stable=True)
    expert = torch.where(torch.isneginf(value), -1, expert)
    return expert[:, :case["topk"]].to(torch.int32).contiguous()


def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    u = z if name == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)
    return z / (1 + torch.exp(-u))


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        u, slope = z, 1.0
    else:
        c = 2 * math.sqrt(2 / math.pi)
        u, slope = c * (z + 0.044715 * z * z * z), c * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-u))
    return s + z * slope * s * (1 - s)


def _run_plain(state):
    case, op = state["case"], state["case"]["op"]
    dtype, direction = DTYPES[case["dtype"]], case["direction"]
    if op == "route":
        expert = _choose(case, state) if direction == "forward" else state["expert"]
        score = _scores(case, state["logits"].float())
        kept, at = expert >= 0, expert.clamp(min=0).long()
        s = torch.where(kept, score.gather(1, at), 0.0)
        total = s.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        if direction == "forward":
            return {"expert": expert, "weight": case["scale"] * (s / total if case["renorm"] else s)}
        g = torch.where(kept, state["d_weight"], 0.0)
        if case["renorm"]:
            g = (g - (g * s).sum(1, keepdim=True) / total) / total
        g = torch.where(kept, case["scale"] * g, 0.0)
        d_score = torch.zeros_like(score).scatter_add_(1, at, g)
        if case["score"] == "softmax":
            d = score * (d_score - (g * s).sum(1, keepdim=True))
        else:
            d = score * _scores(case, -state["logits"].float()) * d_score
        return {"d_logits": d.to(dtype)}
    if op == "norm":
        if direction == "backward":
            r, g = state["x"].float(), state["d_out"].float()
            hat = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS)
            gw = g * state["weight"].float()
            d = torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * (gw - hat * (gw * hat).mean(1, keepdim=True))
            if state["residual"] is not None:
                d = d + state["residual"].float()
            return {"d_x": d.to(dtype), "d_weight": (g * hat).sum(0)}
        out, r = {}, state["x"]
        if state["residual"] is not None:
            r = out["residual"] = (r.float() + state["residual"].float()).to(dtype)
        if direction == "forward":
            r = r.float()
            out["out"] = (r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * state["weight"].float()).to(dtype)
            return out
        # in 64 bits: a block whose largest value is next to a power of two times 448 has one scale or the other
        m, h = r.shape
        inv = torch.rsqrt(r.double().square().mean(1, keepdim=True) + EPS)
        rw = r.float() * state["weight"].float()
        pad = torch.nn.functional.pad(rw, (0, -h % 128)).view(m, -1, 128)
        part, power = torch.frexp(pad.abs().amax(2).double() * inv / E4M3_MAX)
        power = torch.where(part == 0.5, power - 1, power).clamp(min=-126)
        scale = torch.where(part == 0, 1.0, ((power + 127) << 23).to(torch.int32).view(torch.float32))
        y = rw * inv.float() / scale.repeat_interleave(128, 1)[:, :h]
        out["q"], out["scale"] = y.to(torch.float8_e4m3fn), scale
        return out
    if direction == "forward":
        b = state["b"].float()
        z = state["a"].float() @ (b.t() if case["layout"] == "nk" else b)
        if state["bias"] is not None:
            z = z + state["bias"].float()
        out = {"out": (_act(case["act"], z) + state["residual"].float()).to(dtype)}
        if case["save"]:
            out["z"] = z.to(dtype)
        return out
    if case["act"] == "none":
        return {"bgrad": state["d_out"].float().sum(0)}
    d_z = state["d_out"].float() * _act_grad(case["act"], state["z"].float())
    return {"bgrad": d_z.sum(0), "d_z": d_z.to(dtype)}


# ---------------------------------------------------------------- the definition, in 64 bits
def _exact_route(case, state):
    import numpy as np

    logits = state["logits"].double().cpu().numpy()
    bias = None if state["bias"] is None else state["bias"].double().cpu().numpy()
    t, e = logits.shape
    off = np.isneginf(logits)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if case["score"] == "softmax":
            top = logits.max(1, keepdims=True)
            p = np.where(off, 0.0, np.exp(logits - np.where(np.isneginf(top), 0.0, top)))
            s = p / np.maximum(p.sum(1, keepdims=True), np.finfo(float).tiny)
            rest = 1 - s
        else:
            s, rest = 1 / (1 + np.exp(-logits)), 1 / (1 + np.exp(logits))
    if case["direction"] == "backward":
        expert = state["expert"].cpu().numpy().astype(np.int64)
    else:
        key = np.where(off, -np.inf, s + bias) if bias is not None else logits
        if case["groups"] > 1:
            by_sum = np.where(off, -np.inf, s) if bias is None and case["best"] == 2 else key
            parts = np.sort(by_sum.reshape(t, case["groups"], -1), 2)[:, :, ::-1]
            total = parts[:, :, 0].copy()
            if case["best"] == 2 and parts.shape[2] > 1:
                total += np.where(np.isneginf(parts[:, :, 1]), 0.0, parts[:, :, 1])
            gone = np.argsort(-total, 1, kind="stable")[:, case["topk_groups"]:]
            for row, groups in enumerate(gone):
                key[row].reshape(case["groups"], -1)[groups] = -np.inf
        expert = np.argsort(-key, 1, kind="stable")[:, :case["topk"]]
        expert = np.where(np.isneginf(np.take_along_axis(key, expert, 1)), -1, expert)
    kept, rows = expert >= 0, np.arange(t)[:, None]
    chosen = np.where(kept, s[rows, expert], 0.0)
    total = chosen.sum(1, keepdims=True)
    total[total == 0] = 1.0
    if case["direction"] == "forward":
        weight = case["scale"] * chosen / (total if case["renorm"] else 1.0)
        return {"expert": torch.from_numpy(expert.astype(np.int32)), "weight": torch.from_numpy(weight)}
    g = np.where(kept, state["d_weight"].double().cpu().numpy(), 0.0)
    if case["renorm"]:
        g = np.where(kept, g - (g * chosen).sum(1, keepdims=True) / total, 0.0) / total
    d = np.zeros_like(s)
    np.add.at(d, (np.broadcast_to(rows, expert.shape)[kept], expert[kept]), case["scale"] * g[kept])
    if case["score"] == "softmax":
        d = s * (d - (d * s).sum(1, keepdims=True))
    else:
        d = d * s * rest
    return {"d_logits": torch.from_numpy(d)}


def exact(case, seed):
    state = prepare(case, seed)
    op, direction = case["op"], case["direction"]
    if op == "route":
        return _exact_route(case, state)
    if op == "norm":
        x, w = state["x"].double(), state["weight"].double()
        m, h = x.shape
        if direction == "backward":
            inv = (x.square().sum(1) / h + EPS) ** -0.5
            hat = x * inv[:, None]
            dy = state["d_out"].double()
            mean = torch.linalg.vecdot(dy * w, hat) / h
            d = (dy * w - hat * mean[:, None]) * inv[:, None]
            if state["residual"] is not None:
                d += state["residual"].double()
            return {"d_x": d, "d_weight": torch.einsum("mh,mh->h", dy, hat)}
        out = {}
        if state["residual"] is not None:
            out["residual"] = x + state["residual"].double()
            x = out["residual"].to(DTYPES[case["dtype"]]).double()  # the norm is of the stream as it is stored
        y = x * ((x.square().sum(1) / h + EPS) ** -0.5)[:, None] * w
        if direction == "forward":
            out["out"] = y
            return out
        out["q"] = torch.empty_like(y)
        out["scale"] = torch.ones(m, _ceil(h, 128), dtype=torch.float64, device="cuda")
        for j in range(out["scale"].shape[1]):
            part = y[:, 128 * j:128 * j + 128]
            top = part.abs().amax(1)
            power = torch.ceil(torch.log2(top / E4M3_MAX))
            power = torch.where(torch.exp2(power - 1) * E4M3_MAX >= top, power - 1, power)
            s = torch.where(top > 0, torch.exp2(power.clamp(min=-126)), 1.0)
            v = part / s[:, None]
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
            out["scale"][:, j] = s
            out["q"][:, 128 * j:128 * j + 128] = torch.round(v / step) * step
        return out
    bias = 0.0 if state["bias"] is None else state["bias"].double()
    gelu = math.sqrt(2 / math.pi)
    if direction == "forward":
        b = state["b"].double()
        z = state["a"].double() @ (b.t() if case["layout"] == "nk" else b) + bias
        del b
        if case["act"] == "relu":
            y = z.clamp(min=0)
        elif case["act"] == "gelu":
            y = 0.5 * z * (1 + torch.tanh(gelu * (z + 0.044715 * z ** 3)))
        else:
            y = z * torch.sigmoid(z) if case["act"] == "silu" else z
        out = {"out": y + state["residual"].double()}
        if case["save"]:
            out["z"] = z
        return out
    dy = state["d_out"].double()
    if case["act"] == "none":
        return {"bgrad": dy.sum(0)}
    z = state["z"].double()
    if case["act"] == "relu":
        d_z = torch.where(z > 0, dy, 0.0)
    elif case["act"] == "silu":
        d_z = dy * torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    else:
        th = torch.tanh(gelu * (z + 0.044715 * z ** 3))
        d_z = dy * (0.5 * (1 + th) + 0.5 * z * (1 - th * th) * gelu * (1 + 3 * 0.044715 * z * z))
    return {"bgrad": d_z.sum(0), "d_z": d_z}
