"""Mixture-of-experts routing and 8-bit expert products: the cases that are timed, and their plain forms.

Operators, each reached through the package's public entry points:

- dispatch: the (token, slot) pairs of a router's choice are sorted by expert, and every token's row is
  copied to its places (``gf_moe_dispatch_execute``; quantised on the way, ``gf_moe_dispatch_fp8_execute``;
  backward, ``gf_moe_dispatch_grad_execute``).
- combine: each token's rows come back, weighted and summed (``gf_moe_combine_execute``, backward
  ``gf_moe_combine_grad_execute``).
- quantize: e4m3 values with one fp32 scale for each 1 x 128 or 128 x 128 block (``gf_fp8_quantize``).
- matmul: out = A B^T with both operands e4m3 and a scale for each block of 128 (``gf_fp8_matmul_*``).
- experts: the rows of each expert through its gate+up product, SwiGLU, quantisation and its down product
  (two grouped ``gf_fp8_matmul_*`` calls).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token of a serving loop: nothing but latency
        dict(name="dispatch-token", op="dispatch", direction="forward", tokens=1, topk=8, experts=128, hidden=5120, dtype="bf16", drop=0.0),
        # a training step's micro-batch, with a capacity that drops a few slots
        dict(name="dispatch-train", op="dispatch", direction="forward", tokens=16384, topk=8, experts=128, hidden=4096, dtype="bf16", drop=0.01),
        # its gradient, at a width that no vector load divides
        dict(name="dispatch-grad-odd", op="dispatch", direction="backward", tokens=5003, topk=6, experts=60, hidden=2047, dtype="fp16", drop=0.0),
        # a prompt in serving: rows quantised on their way to the experts
        dict(name="dispatch-fp8-prompt", op="dispatch", direction="fp8", tokens=4096, topk=8, experts=128, hidden=5120, dtype="bf16", drop=0.0),
        # a batch of single tokens in serving
        dict(name="combine-decode", op="combine", direction="forward", tokens=64, topk=8, experts=128, hidden=5120, dtype="bf16", drop=0.0),
        # a training step's gradient of the rows and of the router's weights
        dict(name="combine-grad-train", op="combine", direction="backward", tokens=16384, topk=8, experts=128, hidden=4096, dtype="bf16", drop=0.01),
        # activations of a few tokens before a product
        dict(name="quantize-rows-small", op="quantize", rows=16, cols=2048, block_rows=1, dtype="fp16"),
        # a weight laid out once, the MLP's gate projection
        dict(name="quantize-weight", op="quantize", rows=17408, cols=5120, block_rows=128, dtype="bf16"),
        # one token through the MLP's gate projection: the weight is read once
        dict(name="matmul-token", op="matmul", m=1, n=17408, k=5120, dtype="bf16"),
        # a prompt through a wide projection
        dict(name="matmul-prompt", op="matmul", m=8192, n=16384, k=4096, dtype="bf16"),
        # a batch of single tokens over many experts: a few rows each, every weight read once
        dict(name="experts-decode", op="experts", tokens=32, topk=8, experts=128, hidden=2048, inner=1024, dtype="bf16", drop=0.0),
        # a prompt over the experts: some hundred rows each
        dict(name="experts-prompt", op="experts", tokens=4096, topk=8, experts=64, hidden=4096, inner=2048, dtype="bf16", drop=0.0),
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
    op = rng.choice(("dispatch", "combine", "quantize", "matmul", "experts"))
    dtype = rng.choice(("bf16", "fp16"))
    if op in ("dispatch", "combine"):
        direction = rng.choice(("forward", "backward", "fp8") if op == "dispatch" else ("forward", "backward"))
        experts = _log(rng, 4, 256)
        topk = rng.randint(1, min(8, experts))
        hidden = 16 * _log(rng, 8, 512)
        if direction != "fp8":
            hidden += rng.choice((0, 0, 0, 1, 6, 8))
        return dict(op=op, direction=direction, tokens=_log(rng, 1, 16384), topk=topk, experts=experts, hidden=hidden,
                    dtype=dtype, drop=rng.choice((0.0, 0.0, 0.02, 0.3)))
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 17408), cols=16 * _log(rng, 1, 1088), block_rows=rng.choice((1, 128)), dtype=dtype)
    if op == "matmul":
        return dict(op=op, m=_log(rng, 1, 8192), n=8 * _log(rng, 16, 2176), k=16 * _log(rng, 16, 1088), dtype=dtype)
    experts = _log(rng, 4, 128)
    return dict(op=op, tokens=_log(rng, 1, 4096), topk=rng.randint(1, min(8, experts)), experts=experts,
                hidden=16 * _log(rng, 16, 256), inner=16 * _log(rng, 8, 128), dtype=dtype, drop=rng.choice((0.0, 0.0, 0.05)))


def _ceil(a, b):
    return -(-a // b)


def work(case):
    """Each input read once, each output written once; one pass of arithmetic."""
    op = case["op"]
    if op in ("dispatch", "combine"):
        t, k, h = case["tokens"], case["topk"], case["hidden"]
        index, x, rows = t * k * 4, t * h * 2, t * k * h * 2
        if op == "dispatch" and case["direction"] == "forward":
            return {"bytes": 3 * index + x + rows, "flops": 0}
        if op == "dispatch" and case["direction"] == "fp8":
            return {"bytes": 3 * index + x + rows // 2 + t * k * _ceil(h, 128) * 4, "flops": 3 * t * h}
        if op == "dispatch":
            return {"bytes": index + rows + x, "flops": t * k * h}
        if case["direction"] == "forward":
            return {"bytes": 2 * index + rows + x, "flops": 2 * t * k * h}
        return {"bytes": 3 * index + 2 * rows + x, "flops": 3 * t * k * h}
    if op == "quantize":
        m, k = case["rows"], case["cols"]
        return {"bytes": 3 * m * k + _ceil(m, case["block_rows"]) * _ceil(k, 128) * 4, "flops": 3 * m * k}
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        scales = (m + _ceil(n, 128)) * _ceil(k, 128) * 4
        return {"bytes": m * k + n * k + 2 * m * n + scales, "flops": 2 * m * n * k}
    t, k, e, h, i = case["tokens"], case["topk"], case["experts"], case["hidden"], case["inner"]
    r = t * k * (1 - case["drop"])
    used = e * (1 - (1 - 1 / e) ** r)  # experts that any row chose
    return {"bytes": r * (3 * h + h / 32) + used * 3 * h * i * (1 + 4 / 16384), "flops": 6 * r * h * i}


# ---------------------------------------------------------------- the inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _routing(case, gen):
    """A router's choice: distinct experts a token, some experts liked more than others, a few slots dropped (-1)."""
    t, k, e = case["tokens"], case["topk"], case["experts"]
    logits = _randn(gen, t, e) + 0.2 * _randn(gen, e)
    value, expert = torch.topk(logits, k, dim=1)
    weight = torch.softmax(value, dim=1)
    expert = expert.to(torch.int32)
    if case["drop"]:
        expert[torch.rand(t, k, generator=gen, device="cuda") < case["drop"]] = -1
    return expert.contiguous(), weight.contiguous()


def _activations(gen, rows, cols, dtype):
    """Hidden states: rows of different size, a few channels much larger than the rest."""
    x = _randn(gen, rows, cols) * torch.exp(0.5 * _randn(gen, rows, 1)) * torch.exp(0.5 * _randn(gen, 1, cols))
    return x.to(dtype)


def _weights(gen, groups, n, k):
    """e4m3 weights with a scale for each 128 x 128 block, the block's largest magnitude at the type's."""
    q = torch.empty(groups, n, k, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(groups, _ceil(n, 128), _ceil(k, 128), device="cuda")
    step = max(1, (1 << 27) // (n * k))
    for g in range(0, groups, step):
        w = _randn(gen, min(step, groups - g), n, k) / math.sqrt(k)
        amax = _block_max(w, 128)
        s[g:g + step] = amax / E4M3_MAX
        q[g:g + step] = (w / _spread(s[g:g + step], n, k, 128)).to(torch.float8_e4m3fn)
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    state = {"case": case}
    if op in ("dispatch", "combine"):
        t, k, e, h = case["tokens"], case["topk"], case["experts"], case["hidden"]
        state["expert"], state["weight"] = _routing(case, gen)
        if op == "dispatch" and case["direction"] != "backward":
            state["x"] = _activations(gen, t, h, dtype)
        else:
            state["offsets"], state["row_of"], _ = _sort(state["expert"], e)
            state["rows"] = _activations(gen, t * k, h, dtype)
            if op == "combine" and case["direction"] == "backward":
                state["d_out"] = _activations(gen, t, h, dtype)
    elif op == "quantize":
        state["x"] = _activations(gen, case["rows"], case["cols"], dtype)
    elif op == "matmul":
        state["a"], state["a_scale"] = _quantize(_activations(gen, case["m"], case["k"], dtype), 1)
        state["b"], state["b_scale"] = (w[0] for w in _weights(gen, 1, case["n"], case["k"]))
    else:
        e, h, i = case["experts"], case["hidden"], case["inner"]
        expert, _ = _routing(case, gen)
        state["offsets"], _, _ = _sort(expert, e)
        state["most"] = int((state["offsets"][1:] - state["offsets"][:-1]).max())
        state["x"], state["x_scale"] = _quantize(_activations(gen, expert.numel(), h, dtype), 1)
        state["gate"], state["gate_scale"] = _weights(gen, e, i, h)
        state["up"], state["up_scale"] = _weights(gen, e, i, h)
        state["down"], state["down_scale"] = _weights(gen, e, h, i)
    if own:
        _plan(state)
    return state


def _plan(state):
    """The plans and the output buffers that a program keeps from step to step."""
    import gemm_epilogue_tmem_gb300 as gf

    case, op = state["case"], state["case"]["op"]
    dtype = DTYPES[case["dtype"]]
    code = gf.GF_BF16 if case["dtype"] == "bf16" else gf.GF_F16

    def new(*shape, dtype=dtype):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op in ("dispatch", "combine"):
        t, k, e, h = case["tokens"], case["topk"], case["experts"], case["hidden"]
        state["plan"] = gf.gf_moe_plan(t, k, e, h, code)
        if op == "dispatch" and case["direction"] != "backward":
            fp8 = case["direction"] == "fp8"
            out = {"offsets": new(e + 1, dtype=torch.int32), "row_of": new(t, k, dtype=torch.int32), "slot_of": new(t * k, dtype=torch.int32),
                   "rows": new(t * k, h, dtype=torch.float8_e4m3fn if fp8 else dtype)}
            if fp8:
                out["scale"] = new(t * k, _ceil(h, 128), dtype=torch.float32)
        elif op == "dispatch":
            out = {"d_x": new(t, h)}
        elif case["direction"] == "forward":
            out = {"out": new(t, h)}
        else:
            out = {"d_rows": new(t * k, h), "d_weight": new(t, k, dtype=torch.float32)}
    elif op == "quantize":
        m, k = case["rows"], case["cols"]
        out = {"q": new(m, k, dtype=torch.float8_e4m3fn), "scale": new(_ceil(m, case["block_rows"]), _ceil(k, 128), dtype=torch.float32)}
        state["code"] = code
    elif op == "matmul":
        state["plan"] = gf.gf_fp8_matmul_plan(case["m"], case["n"], case["k"], 1, code, gf.GF_FP8_EPILOG_NONE)
        out = {"out": new(case["m"], case["n"])}
    else:
        r, e, h, i = case["tokens"] * case["topk"], case["experts"], case["hidden"], case["inner"]
        state["plan"] = gf.gf_fp8_matmul_plan(r, i, h, e, code, gf.GF_FP8_EPILOG_SWIGLU_QUANT)
        state["plan_down"] = gf.gf_fp8_matmul_plan(r, h, i, e, code, gf.GF_FP8_EPILOG_NONE)
        state["h"], state["h_scale"] = new(r, i, dtype=torch.float8_e4m3fn), new(r, _ceil(i, 128), dtype=torch.float32)
        out = {"out": new(r, h)}
    state["out"] = out


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import gemm_epilogue_tmem_gb300 as gf

    case, out = state["case"], state["out"]
    op, direction = case["op"], case.get("direction")
    if op == "dispatch" and direction == "forward":
        gf.gf_moe_dispatch_execute(state["plan"], state["expert"], state["x"], out["offsets"], out["row_of"], out["slot_of"], out["rows"])
    elif op == "dispatch" and direction == "fp8":
        gf.gf_moe_dispatch_fp8_execute(state["plan"], state["expert"], state["x"], out["offsets"], out["row_of"], out["slot_of"], out["rows"], out["scale"])
    elif op == "dispatch":
        gf.gf_moe_dispatch_grad_execute(state["plan"], state["row_of"], state["rows"], out["d_x"])
    elif op == "combine" and direction == "forward":
        gf.gf_moe_combine_execute(state["plan"], state["row_of"], state["weight"], state["rows"], out["out"])
    elif op == "combine":
        gf.gf_moe_combine_grad_execute(state["plan"], state["offsets"], state["row_of"], state["weight"], state["rows"], state["d_out"], out["d_rows"], out["d_weight"])
    elif op == "quantize":
        gf.gf_fp8_quantize(case["rows"], case["cols"], state["code"], case["block_rows"], state["x"], out["q"], out["scale"])
    elif op == "matmul":
        gf.gf_fp8_matmul_execute(state["plan"], state["a"], state["a_scale"], state["b"], state["b_scale"], out=out["out"])
    else:
        gf.gf_fp8_matmul_execute(state["plan"], state["x"], state["x_scale"], state["gate"], state["gate_scale"], state["up"], state["up_scale"],
                                 offsets=state["offsets"], out=state["h"], out_scale=state["h_scale"])
        gf.gf_fp8_matmul_execute(state["plan_down"], state["h"], state["h_scale"], state["down"], state["down_scale"],
                                 offsets=state["offsets"], out=out["out"])
    return out


# ---------------------------------------------------------------- the plain forms
def _sort(expert, experts):
    """Slots by expert, in the slots' own order within one; dropped slots (an id outside the experts) last, without a row."""
    flat = expert.reshape(-1)
    key = torch.where((flat < 0) | (flat >= experts), experts, flat)
    slot_of = torch.argsort(key, stable=True)
    row_of = torch.empty_like(slot_of)
    row_of[slot_of] = torch.arange(flat.numel(), device=flat.device)
    offsets = torch.searchsorted(key[slot_of], torch.arange(experts + 1, device=flat.device, dtype=key.dtype))
    row_of = torch.where(key < experts, row_of, -1)
    slot_of = torch.where(key[slot_of] < experts, slot_of, -1)
    return offsets.to(torch.int32), row_of.to(torch.int32).reshape(expert.shape), slot_of.to(torch.int32)


def _block_max(x, block_rows):
    """The largest magnitude of each block of block_rows x 128, over the last two dimensions."""
    n, k = x.shape[-2:]
    pad = torch.nn.functional.pad(x.abs(), (0, -k % 128, 0, -n % block_rows))
    return pad.unflatten(-1, (-1, 128)).unflatten(-3, (-1, block_rows)).amax(dim=(-3, -1))


def _spread(s, n, k, block_rows):
    """Each block's scale over its elements: s [..., ceil(n / block_rows), ceil(k / 128)] -> [..., n, k]."""
    wide = s[..., :, None, :, None].expand(*s.shape[:-1], block_rows, s.shape[-1], 128)
    return wide.flatten(-2).flatten(-3, -2)[..., :n, :k]


def _quantize(x, block_rows):
    """e4m3 values and scales: the smallest power of two that brings the block's largest magnitude to 448 or less, 1 for a block of zeros."""
    x = x.float()
    amax = _block_max(x, block_rows)
    part, power = torch.frexp(amax / E4M3_MAX)
    power = torch.where(part == 0.5, power - 1, power)
    scale = torch.where(amax == 0, 1.0, ((power.clamp(min=-126) + 127) << 23).view(torch.float32))
    return (x / _spread(scale, *x.shape, block_rows)).to(torch.float8_e4m3fn), scale


def _run_plain(state):
    case = state["case"]
    op, direction, dtype = case["op"], case.get("direction"), DTYPES[case["dtype"]]
    if op in ("dispatch", "combine"):
        t, k, h = case["tokens"], case["topk"], case["hidden"]
        if op == "dispatch" and direction != "backward":
            offsets, row_of, slot_of = _sort(state["expert"], case["experts"])
            token, kept = slot_of.clamp(min=0) // k, slot_of >= 0
            out = {"offsets": offsets, "row_of": row_of, "slot_of": slot_of}
            if direction == "fp8":
                q, scale = _quantize(state["x"], 1)
                out["rows"] = torch.where(kept[:, None], q.view(torch.uint8)[token], 0).view(torch.float8_e4m3fn)
                out["scale"] = torch.where(kept[:, None], scale[token], 1.0)
            else:
                out["rows"] = torch.where(kept[:, None], state["x"][token], 0)
            return out
        kept = state["row_of"] >= 0
        at = state["row_of"].clamp(min=0)
        if op == "dispatch":
            return {"d_x": (state["rows"][at].float() * kept[:, :, None]).sum(1).to(dtype)}
        weight = state["weight"] * kept
        if direction == "forward":
            return {"out": (state["rows"][at].float() * weight[:, :, None]).sum(1).to(dtype)}
        d_out = state["d_out"].float()
        d_weight = (state["rows"][at].float() * d_out[:, None, :]).sum(2) * kept
        d_rows = torch.zeros(t * k + 1, h, dtype=dtype, device=d_out.device)
        d_rows[torch.where(kept, at, t * k).reshape(-1)] = (weight[:, :, None] * d_out[:, None, :]).to(dtype).reshape(t * k, h)
        return {"d_rows": d_rows[: t * k], "d_weight": d_weight}
    if op == "quantize":
        q, scale = _quantize(state["x"], case["block_rows"])
        return {"q": q, "scale": scale}
    if op == "matmul":
        a = state["a"].float() * _spread(state["a_scale"], *state["a"].shape, 1)
        b = state["b"].float() * _spread(state["b_scale"], *state["b"].shape, 128)
        return {"out": (a @ b.t()).to(dtype)}
    e, h, i, most = case["experts"], case["hidden"], case["inner"], state["most"]
    r = state["x"].shape[0]
    row = torch.arange(r, device="cuda")
    group = torch.searchsorted(state["offsets"][1:].contiguous(), row, right=True)
    kept = group < e
    group = group.clamp(max=e - 1)
    place = torch.where(kept, row - state["offsets"][group], most)

    def product(x, w, s):
        """The rows of each group times its weight, over groups padded to one length."""
        n, k = w.shape[1:]
        padded = torch.zeros(e, most + 1, k, device="cuda")
        padded[group, place] = x * kept[:, None]
        return torch.bmm(padded, (w.float() * _spread(s, n, k, 128)).transpose(1, 2))[group, place] * kept[:, None]

    x = state["x"].float() * _spread(state["x_scale"], r, h, 1)
    g = product(x, state["gate"], state["gate_scale"])
    u = product(x, state["up"], state["up_scale"])
    q, scale = _quantize(g / (1 + torch.exp(-g)) * u, 1)
    return {"out": product(q.float() * _spread(scale, r, i, 1), state["down"], state["down_scale"]).to(dtype)}


# ---------------------------------------------------------------- the definition, in 64 bits
def _values(q, scale, block_rows):
    rows = torch.arange(q.shape[0], device="cuda") // block_rows
    cols = torch.arange(q.shape[1], device="cuda") // 128
    return q.double() * scale.double()[rows][:, cols]


def _to_e4m3(v):
    """Values of magnitude at most 448 rounded to e4m3 (three bits after the leading one, none below 2^-9), ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _blocks64(x, block_rows):
    """(e4m3 values, scales) of a matrix in 64 bits."""
    m, k = x.shape
    scale = torch.ones(_ceil(m, block_rows), _ceil(k, 128), dtype=torch.float64, device="cuda")
    q = torch.empty_like(x)
    for j in range(scale.shape[1]):
        part = x[:, 128 * j:128 * j + 128]
        top = part.abs().amax(1)
        if block_rows > 1:
            top = torch.stack([p.amax() for p in top.split(block_rows)])
        power = torch.ceil(torch.log2(top / E4M3_MAX))
        power = torch.where(torch.exp2(power - 1) * E4M3_MAX >= top, power - 1, power)
        s = torch.where(top > 0, torch.exp2(power.clamp(min=-126)), 1.0)
        scale[:, j] = s
        q[:, 128 * j:128 * j + 128] = _to_e4m3(part / s.repeat_interleave(block_rows)[:m, None])
    return q, scale


def exact(case, seed):
    state = prepare(case, seed)
    op, direction = case["op"], case.get("direction")
    if op in ("dispatch", "combine"):
        t, k, e, h = case["tokens"], case["topk"], case["experts"], case["hidden"]
        choice = state["expert"].reshape(-1).cpu().tolist()
        slots = [[] for _ in range(e)]
        for slot, at in enumerate(choice):
            if 0 <= at < e:
                slots[at].append(slot)
        order = [slot for part in slots for slot in part]
        at = torch.tensor(order, dtype=torch.int64, device="cuda")
        rows = torch.arange(len(order), device="cuda")
        if op == "dispatch" and direction != "backward":
            offsets = [0]
            for part in slots:
                offsets.append(offsets[-1] + len(part))
            row_of = torch.full((t * k,), -1, dtype=torch.int32, device="cuda")
            row_of[at] = rows.to(torch.int32)
            slot_of = torch.full((t * k,), -1, dtype=torch.int32, device="cuda")
            slot_of[rows] = at.to(torch.int32)
            out = {"offsets": torch.tensor(offsets, dtype=torch.int32), "row_of": row_of.reshape(t, k), "slot_of": slot_of}
            x = state["x"].double()
            if direction == "fp8":
                x, scale = _blocks64(x, 1)
                out["scale"] = torch.ones(t * k, scale.shape[1], dtype=torch.float64, device="cuda")
                out["scale"][rows] = scale[at // k]
            out["rows"] = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
            out["rows"][rows] = x[at // k]
            return out
        token, values = at // k, state["rows"][: len(order)]
        weight = state["weight"].double().reshape(-1)[at]
        if direction == "forward" or op == "dispatch":
            out = torch.zeros(t, h, dtype=torch.float64, device="cuda")
            out.index_add_(0, token, values.double() * (weight[:, None] if op == "combine" else 1.0))
            return {"d_x" if op == "dispatch" else "out": out}
        d_out = state["d_out"].double()
        d_weight = torch.zeros(t * k, dtype=torch.float64, device="cuda")
        d_weight[at] = torch.linalg.vecdot(values.double(), d_out[token])
        d_rows = torch.zeros(t * k, h, dtype=torch.float64, device="cuda")
        d_rows[rows] = weight[:, None] * d_out[token]
        return {"d_rows": d_rows, "d_weight": d_weight.reshape(t, k)}
    if op == "quantize":
        q, scale = _blocks64(state["x"].double(), case["block_rows"])
        return {"q": q, "scale": scale}
    if op == "matmul":
        return {"out": _values(state["a"], state["a_scale"], 1) @ _values(state["b"], state["b_scale"], 128).t()}
    ends = state["offsets"].cpu().tolist()
    out = torch.zeros(state["x"].shape[0], case["hidden"], dtype=torch.float64, device="cuda")
    for e, (first, last) in enumerate(zip(ends[:-1], ends[1:])):
        x = _values(state["x"][first:last], state["x_scale"][first:last], 1)
        g = x @ _values(state["gate"][e], state["gate_scale"][e], 128).t()
        u = x @ _values(state["up"][e], state["up_scale"][e], 128).t()
        if last > first:
            q, scale = _blocks64(g * torch.sigmoid(g) * u, 1)
            wide = scale.repeat_interleave(128, 1)[:, : q.shape[1]]
            out[first:last] = (q * wide) @ _values(state["down"][e], state["down_scale"][e], 128).t()
    return {"out": out}
