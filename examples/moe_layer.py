"""A mixture-of-experts layer on the library's routing and products.

Serving (``MoeLayer.serve``): the router's logits by ``gf_matmul``, its choice,
``gf_moe_dispatch_fp8`` (sort, quantise, copy), the experts' gate+up product
with SwiGLU and quantisation and their down product (``gf_fp8_matmul``), and
``gf_moe_combine``. Nothing is read back to the host.

The gradients (``MoeLayer.train``): the same routing on 16-bit rows, each expert's
SwiGLU through ``gf_swiglu`` / ``gf_dswiglu``, and the gradients of the input
and of the router's weights through ``gf_moe_combine_grad`` and
``gf_moe_dispatch_grad``. The experts' weights are held: their gradients, and 16-bit
products over groups of rows, are not among the library's operators, so that the
experts' numbers of rows are read back and each has products of its own.

    python examples/moe_layer.py [tokens]
"""
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import gemm_epilogue_tmem_gb300 as gf  # noqa: E402


def _empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class MoeLayer:
    def __init__(self, hidden=2048, inner=1024, experts=32, topk=4, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.inner, self.experts, self.topk = hidden, inner, experts, topk

        def weight(*shape):
            w = torch.randn(*shape, generator=gen, device="cuda") / shape[-1] ** 0.5
            return w.bfloat16()

        # gf_matmul takes columns by eights: rows of zeros behind the experts'
        self.router = torch.zeros(-(-experts // 8) * 8, hidden, dtype=torch.bfloat16, device="cuda")
        self.router[:experts] = weight(experts, hidden)
        self.gate, self.up = weight(experts, inner, hidden), weight(experts, inner, hidden)
        self.down = weight(experts, hidden, inner)
        self.fp8 = {name: self._quantized(getattr(self, name)) for name in ("gate", "up", "down")}
        self.plans = {}  # by number of tokens: a serving program keeps a plan for each batch size
        self.expert_plans = {}  # by product and number of rows

    def _quantized(self, w):
        """The experts' weights in e4m3, a scale for each 128 x 128 block."""
        e, n, k = w.shape
        q = _empty(e, n, k, dtype=torch.uint8)
        s = _empty(e, -(-n // 128), -(-k // 128), dtype=torch.float32)
        for i in range(e):
            gf.gf_fp8_quantize(n, k, gf.GF_BF16, 128, w[i], q[i], s[i])
        return q, s

    def _kept(self, tokens):
        """Plans and buffers for this many tokens."""
        if tokens in self.plans:
            return self.plans[tokens]
        h, i, e, slots = self.hidden, self.inner, self.experts, tokens * self.topk
        p = {
            "router": gf.gf_matmul_plan_ex(tokens, len(self.router), h, gf.GF_BF16, gf.GF_EPILOG_NONE, gf.GF_BIAS_COL, gf.GF_B_NK),
            "moe": gf.gf_moe_plan(tokens, self.topk, e, h, gf.GF_BF16),
            "gate_up": gf.gf_fp8_matmul_plan(slots, i, h, e, gf.GF_BF16, gf.GF_FP8_EPILOG_SWIGLU_QUANT),
            "down": gf.gf_fp8_matmul_plan(slots, h, i, e, gf.GF_BF16),
            "logits": _empty(tokens, len(self.router)),
            "offsets": _empty(e + 1, dtype=torch.int32), "slot_of": _empty(slots, dtype=torch.int32),
            "row_of": _empty(tokens, self.topk, dtype=torch.int32),
            "rows8": _empty(slots, h, dtype=torch.uint8), "scale": _empty(slots, -(-h // 128), dtype=torch.float32),
            "h8": _empty(slots, i, dtype=torch.uint8), "h_scale": _empty(slots, -(-i // 128), dtype=torch.float32),
            "rows": _empty(slots, h), "out": _empty(tokens, h),
        }
        self.plans[tokens] = p
        return p

    def _expert_plan(self, product, rows):
        """The plan of one expert's 16-bit product. Kept: a plan may be freed only when its work is done."""
        key = product, rows
        if key not in self.expert_plans:
            h, i, bf16 = self.hidden, self.inner, gf.GF_BF16
            self.expert_plans[key] = {
                "gate_up": lambda: gf.gf_swiglu_plan(rows, i, h, bf16, save_gu=True),
                "down": lambda: gf.gf_matmul_plan_ex(rows, h, i, bf16, gf.GF_EPILOG_NONE, gf.GF_BIAS_COL, gf.GF_B_NK),
                "d_hid": lambda: gf.gf_dswiglu_plan(rows, i, h, bf16),
                "d_rows": lambda: gf.gf_matmul_plan(rows, h, i, bf16, gf.GF_EPILOG_NONE),
            }[product]()
        return self.expert_plans[key]

    def route(self, x, p):
        """The router's choice: experts and weights of each token."""
        gf.gf_matmul_execute(p["router"], x, self.router, out=p["logits"])
        value, expert = torch.topk(p["logits"][:, :self.experts].float(), self.topk, dim=1)
        return expert.to(torch.int32), torch.softmax(value, dim=1)

    def serve(self, x):
        p = self._kept(x.shape[0])
        expert, weight = self.route(x, p)
        gf.gf_moe_dispatch_fp8_execute(p["moe"], expert, x, p["offsets"], p["row_of"], p["slot_of"],
                                       p["rows8"], p["scale"])
        gf.gf_fp8_matmul_execute(p["gate_up"], p["rows8"], p["scale"], *self.fp8["gate"], *self.fp8["up"],
                                 offsets=p["offsets"], out=p["h8"], out_scale=p["h_scale"])
        gf.gf_fp8_matmul_execute(p["down"], p["h8"], p["h_scale"], *self.fp8["down"],
                                 offsets=p["offsets"], out=p["rows"])
        gf.gf_moe_combine_execute(p["moe"], p["row_of"], weight, p["rows"], p["out"])
        return p["out"]

    def train(self, x, d_out):
        """(out, d_x, d_weight): forward, and the gradients of the input (through
        the experts, the router's choice held) and of the router's weights."""
        p = self._kept(x.shape[0])
        h, i = self.hidden, self.inner
        expert, weight = self.route(x, p)
        rows, d_rows = p["rows"], torch.empty_like(p["rows"])
        gf.gf_moe_dispatch_execute(p["moe"], expert, x, p["offsets"], p["row_of"], p["slot_of"], rows)
        ends = p["offsets"].tolist()  # the 16-bit plans take their sizes from the host
        y, saved = torch.empty_like(rows), []
        for e in range(self.experts):
            part = slice(ends[e], ends[e + 1])
            n = ends[e + 1] - ends[e]
            hid, g, u = _empty(n, i), _empty(n, i), _empty(n, i)
            gf.gf_swiglu_execute(self._expert_plan("gate_up", n), rows[part].contiguous(), self.gate[e], self.up[e], hid, g, u)
            out = _empty(n, h)
            gf.gf_matmul_execute(self._expert_plan("down", n), hid, self.down[e], out=out)
            y[part] = out
            saved.append((part, n, g, u))
        gf.gf_moe_combine_execute(p["moe"], p["row_of"], weight, y, p["out"])

        d_y, d_weight = torch.empty_like(y), torch.empty_like(weight)
        gf.gf_moe_combine_grad_execute(p["moe"], p["offsets"], p["row_of"], weight, y, d_out, d_y, d_weight)
        for e, (part, n, g, u) in enumerate(saved):
            d_gate, d_up = _empty(n, i), _empty(n, i)
            gf.gf_dswiglu_execute(self._expert_plan("d_hid", n), d_y[part].contiguous(), self.down[e], g, u, d_gate, d_up)
            plan, a, b = self._expert_plan("d_rows", n), _empty(n, h), _empty(n, h)
            gf.gf_matmul_execute(plan, d_gate, self.gate[e], out=a)
            gf.gf_matmul_execute(plan, d_up, self.up[e], out=b)
            d_rows[part] = a + b
        d_rows[ends[-1]:] = 0
        d_x = torch.empty_like(x)
        gf.gf_moe_dispatch_grad_execute(p["moe"], p["row_of"], d_rows, d_x)
        return p["out"], d_x, d_weight


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 1024
    gf.build()
    layer = MoeLayer()
    x = torch.randn(tokens, layer.hidden, device="cuda").bfloat16()
    out = layer.serve(x).clone()  # the layer keeps its output buffer
    torch.cuda.synchronize()
    start = time.perf_counter()
    for _ in range(20):
        layer.serve(x)
    torch.cuda.synchronize()
    print(f"serve: {tokens} tokens, {(time.perf_counter() - start) / 20 * 1e6:.0f} us a layer")
    exact, _, d_weight = layer.train(x, torch.randn_like(x))
    err = (out.float() - exact.float()).norm() / exact.float().norm()
    print(f"e4m3 against 16-bit experts: relative difference {err:.3f}; d_weight {tuple(d_weight.shape)}")


if __name__ == "__main__":
    main()
