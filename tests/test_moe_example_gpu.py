"""examples/moe_layer.py, the routing and the products run together, against
the same layer in torch, 64 bits."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def layer64(layer, x, expert, weight, weights):
    """The layer in 64 bits on given weights and a given choice."""
    gate, up, down = weights
    out = torch.zeros_like(x)
    for e in range(layer.experts):
        token, slot = torch.nonzero(expert == e, as_tuple=True)
        if token.numel():
            rows = x[token]
            y = (torch.nn.functional.silu(rows @ gate[e].t()) * (rows @ up[e].t())) @ down[e].t()
            out = out.index_add(0, token, weight[token, slot, None] * y)
    return out


@pytest.mark.parametrize("tokens", [1, 37, 600])
def test_serve(example, tokens):
    """Every product sees operands rounded to e4m3: relative errors of up to
    2^-4 each (rms 2^-4 / sqrt(3) = 0.036), of rows and weights in gate and up
    (two products of them), of h and the down weight. Summed as independent
    errors, sqrt(6) * 0.036 = 0.088, below 0.1 in the 2-norm; the bf16 logits
    may order ties otherwise, which the choice that the layer made settles."""
    layer = example.MoeLayer(hidden=512, inner=384, experts=8, topk=2, seed=1)
    x = torch.randn(tokens, 512, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    out = layer.serve(x).clone()
    expert, weight = layer.route(x, layer.plans[tokens])
    want = layer64(layer, x.double(), expert, weight.double(), [w.double() for w in (layer.gate, layer.up, layer.down)])
    assert (out.double() - want).norm() / want.norm() < 0.1
    # and against the quantised weights themselves only the rows and h are rounded:
    # gate and up share the rows' error, h has its own
    deq = []
    for name in ("gate", "up", "down"):
        q, s = layer.fp8[name]
        n, k = q.shape[1:]
        wide = s.double().repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k]
        deq.append(q.view(torch.float8_e4m3fn).double() * wide)
    want = layer64(layer, x.double(), expert, weight.double(), deq)
    assert (out.double() - want).norm() / want.norm() < 0.07
    assert torch.equal(layer.serve(x), out)


def test_train(example):
    """out, d_x and d_weight against 64-bit autograd; g, u, h, y and the
    gradients between the products are rounded to bf16 (2^-8 each, about ten
    of them: well below 2 % in the 2-norm)."""
    layer = example.MoeLayer(hidden=256, inner=384, experts=6, topk=2, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, d_out = (torch.randn(200, 256, generator=gen, device="cuda").bfloat16() for _ in range(2))
    out, d_x, d_weight = layer.train(x, d_out)
    expert, weight = layer.route(x, layer.plans[200])
    x64, w64 = x.double().requires_grad_(), weight.double().requires_grad_()
    want = layer64(layer, x64, expert, w64, [w.double() for w in (layer.gate, layer.up, layer.down)])
    want.backward(d_out.double())
    for got, ref in ((out, want), (d_x, x64.grad), (d_weight, w64.grad)):
        assert (got.double() - ref).norm() / ref.norm() < 2e-2
