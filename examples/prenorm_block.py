"""A pre-norm block on the library: a dense MLP and a mixture of experts that each
read a root-mean-square norm of the residual stream and add to it.

Dense (``DenseBlock``): the norm (``gf_rmsnorm``, which also adds what came before to the
stream), GELU of the first product (``gf_matmul``), and the second product with its
bias and the stream added in the kernel (``gf_matmul_residual``). ``gradients`` goes back
through the same: ``gf_dact_bgrad`` (the last bias), DGELU_BGRAD, ``gf_rmsnorm_grad``.

Experts (``ExpertBlock``): the norm, the router's logits and its choice (``gf_route``: sigmoid
scores, groups of experts, a bias that only the choice sees), dispatch with quantisation, the
e4m3 experts, and combine. ``gradients`` of what the router adds: ``gf_moe_combine_grad``,
``gf_route_grad``, and its product with the experts' gradient added in the kernel.

    python examples/prenorm_block.py [tokens]
"""
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import gemm_epilogue_tmem_gb300 as gf  # noqa: E402

BF16 = gf.GF_BF16


def _empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _weight(gen, *shape):
    return (torch.randn(*shape, generator=gen, device="cuda") / shape[-1] ** 0.5).bfloat16()


class DenseBlock:
    def __init__(self, hidden=2048, inner=8192, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.inner = hidden, inner
        self.norm = (1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")).bfloat16()
        self.w1, self.b1 = _weight(gen, inner, hidden), 0.1 * _weight(gen, 1, inner)[0]
        self.w2, self.b2 = _weight(gen, hidden, inner), 0.1 * _weight(gen, 1, hidden)[0]
        self.plans = {}  # by number of tokens

    def _kept(self, tokens):
        if tokens not in self.plans:
            h, i = self.hidden, self.inner
            self.plans[tokens] = {
                "norm": gf.gf_rmsnorm_plan(tokens, h, BF16),
                "up": gf.gf_matmul_plan_ex(tokens, i, h, BF16, gf.GF_EPILOG_GELU_AUX_BIAS, gf.GF_BIAS_COL, gf.GF_B_NK),
                "down": gf.gf_matmul_residual_plan(tokens, h, i, BF16, gf.GF_ACT_NONE, gf.GF_B_NK),
                "d_b2": gf.gf_dact_bgrad_plan(tokens, h, BF16, gf.GF_ACT_NONE),
                "d_z": gf.gf_matmul_plan_ex(tokens, i, h, BF16, gf.GF_EPILOG_DGELU_BGRAD, gf.GF_BIAS_COL, gf.GF_B_KN),
                "d_y": gf.gf_matmul_plan_ex(tokens, h, i, BF16, gf.GF_EPILOG_NONE, gf.GF_BIAS_COL, gf.GF_B_KN),
                "y": _empty(tokens, h), "hid": _empty(tokens, i), "z": _empty(tokens, i), "r": _empty(tokens, h),
            }
        return self.plans[tokens]

    def forward(self, x, stream):
        """The stream after this block; x is what the block before it adds."""
        p = self._kept(x.shape[0])
        gf.gf_rmsnorm_execute(p["norm"], x, self.norm, residual=stream, residual_out=p["r"], out=p["y"])
        gf.gf_matmul_execute(p["up"], p["y"], self.w1, bias=self.b1, out=p["hid"], aux_out=p["z"])
        out = _empty(*stream.shape)
        gf.gf_matmul_residual_execute(p["down"], p["hid"], self.w2, p["r"], out, bias=self.b2)
        return out

    def gradients(self, d_out):
        """After forward: the gradients of x and the stream (they are equal), of the norm's weight and of the biases."""
        p, tokens = self._kept(d_out.shape[0]), d_out.shape[0]
        d_b1, d_b2, d_norm = (_empty(n, dtype=torch.float32) for n in (self.inner, self.hidden, self.hidden))
        gf.gf_dact_bgrad_execute(p["d_b2"], d_out, bgrad=d_b2)
        d_z, d_y, d_x = _empty(tokens, self.inner), _empty(tokens, self.hidden), _empty(tokens, self.hidden)
        gf.gf_matmul_execute(p["d_z"], d_out, self.w2, out=d_z, aux_in=p["z"], bgrad=d_b1)
        gf.gf_matmul_execute(p["d_y"], d_z, self.w1, out=d_y)
        gf.gf_rmsnorm_grad_execute(p["norm"], d_y, p["r"], self.norm, d_x, d_weight=d_norm, d_residual=d_out)
        return {"x": d_x, "norm": d_norm, "b1": d_b1, "b2": d_b2}


class ExpertBlock:
    def __init__(self, hidden=2048, inner=1024, experts=64, topk=6, groups=8, topk_groups=4, scale=2.5, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.inner, self.experts, self.topk, self.scale = hidden, inner, experts, topk, scale
        self.groups, self.topk_groups = groups, topk_groups
        self.norm = (1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")).bfloat16()
        # gf_matmul takes columns by eights: rows of zeros behind the experts'
        self.router = torch.zeros(-(-experts // 8) * 8, hidden, dtype=torch.bfloat16, device="cuda")
        self.router[:experts] = _weight(gen, experts, hidden)
        self.balance = 0.05 * torch.randn(experts, generator=gen, device="cuda")
        self.gate, self.up = (self._quantized(_weight(gen, experts, inner, hidden)) for _ in range(2))
        self.down = self._quantized(_weight(gen, experts, hidden, inner))
        self.plans = {}

    def _quantized(self, w):
        e, n, k = w.shape
        q, s = _empty(e, n, k, dtype=torch.uint8), _empty(e, -(-n // 128), -(-k // 128), dtype=torch.float32)
        for i in range(e):
            gf.gf_fp8_quantize(n, k, BF16, 128, w[i], q[i], s[i])
        return q, s

    def _kept(self, t):
        if t not in self.plans:
            h, i, e, k, ld = self.hidden, self.inner, self.experts, self.topk, len(self.router)
            self.plans[t] = {
                "norm": gf.gf_rmsnorm_plan(t, h, BF16),
                "router": gf.gf_matmul_plan_ex(t, ld, h, BF16, gf.GF_EPILOG_NONE, gf.GF_BIAS_COL, gf.GF_B_NK),
                "route": gf.gf_route_plan(t, e, k, BF16, gf.GF_SCORE_SIGMOID, renorm=True, scale=self.scale, groups=self.groups,
                                          topk_groups=self.topk_groups, group_best=2, ld=ld),
                "moe": gf.gf_moe_plan(t, k, e, h, BF16),
                "gate_up": gf.gf_fp8_matmul_plan(t * k, i, h, e, BF16, gf.GF_FP8_EPILOG_SWIGLU_QUANT),
                "down": gf.gf_fp8_matmul_plan(t * k, h, i, e, BF16),
                "d_y": gf.gf_matmul_residual_plan(t, h, ld, BF16, gf.GF_ACT_NONE, gf.GF_B_KN),
                "r": _empty(t, h), "y": _empty(t, h), "logits": _empty(t, ld), "d_logits": _empty(t, ld),
                "expert": _empty(t, k, dtype=torch.int32), "weight": _empty(t, k, dtype=torch.float32),
                "offsets": _empty(e + 1, dtype=torch.int32), "row_of": _empty(t, k, dtype=torch.int32), "slot_of": _empty(t * k, dtype=torch.int32),
                "rows8": _empty(t * k, h, dtype=torch.uint8), "scale": _empty(t * k, -(-h // 128), dtype=torch.float32),
                "h8": _empty(t * k, i, dtype=torch.uint8), "h_scale": _empty(t * k, -(-i // 128), dtype=torch.float32),
                "rows": _empty(t * k, h), "out": _empty(t, h),
            }
        return self.plans[t]

    def forward(self, x, stream):
        """(what this block adds to the stream, the stream with x added). Nothing is read back to the host."""
        p = self._kept(x.shape[0])
        gf.gf_rmsnorm_execute(p["norm"], x, self.norm, residual=stream, residual_out=p["r"], out=p["y"])
        gf.gf_matmul_execute(p["router"], p["y"], self.router, out=p["logits"])
        gf.gf_route_execute(p["route"], p["logits"], p["expert"], p["weight"], bias=self.balance)
        gf.gf_moe_dispatch_fp8_execute(p["moe"], p["expert"], p["y"], p["offsets"], p["row_of"], p["slot_of"], p["rows8"], p["scale"])
        gf.gf_fp8_matmul_execute(p["gate_up"], p["rows8"], p["scale"], *self.gate, *self.up, offsets=p["offsets"], out=p["h8"],
                                 out_scale=p["h_scale"])
        gf.gf_fp8_matmul_execute(p["down"], p["h8"], p["h_scale"], *self.down, offsets=p["offsets"], out=p["rows"])
        gf.gf_moe_combine_execute(p["moe"], p["row_of"], p["weight"], p["rows"], p["out"])
        return p["out"], p["r"]

    def gradients(self, d_out, d_experts):
        """After forward: the gradients of the experts' rows, the logits and y, the norm's output; d_experts is what the
        experts themselves pass back to y (a program's own, through its 16-bit weights)."""
        p, t = self._kept(d_out.shape[0]), d_out.shape[0]
        d_rows, d_weight, d_y = _empty(t * self.topk, self.hidden), _empty(t, self.topk, dtype=torch.float32), _empty(t, self.hidden)
        gf.gf_moe_combine_grad_execute(p["moe"], p["offsets"], p["row_of"], p["weight"], p["rows"], d_out, d_rows, d_weight)
        gf.gf_route_grad_execute(p["route"], p["logits"], p["expert"], d_weight, p["d_logits"])
        gf.gf_matmul_residual_execute(p["d_y"], p["d_logits"], self.router, d_experts, d_y)
        return {"rows": d_rows, "weight": d_weight, "logits": p["d_logits"], "y": d_y}


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 2048
    gf.build()
    dense, experts = DenseBlock(), ExpertBlock()
    x, stream = (torch.randn(tokens, dense.hidden, device="cuda").bfloat16() for _ in range(2))

    def step():
        s = dense.forward(x, stream)
        add, s = experts.forward(x, s)
        return dense.forward(add, s)

    step()
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(20):
        step()
    torch.cuda.synchronize()
    print(f"{tokens} tokens, dense + experts + dense: {(time.perf_counter() - start) / 20 * 1e6:.0f} us")
    grads = dense.gradients(torch.randn_like(x))
    print("gradients:", {k: tuple(v.shape) for k, v in grads.items()})


if __name__ == "__main__":
    main()
