"""examples/moe_layer.py keeps its plans: gf_plan_free may be called only when a plan's work has completed."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_epilogue_tmem_gb300 as gf  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_plan_is_freed_under_its_work(monkeypatch):
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer = example.MoeLayer(hidden=256, inner=128, experts=5, topk=2, seed=1)
    x = torch.randn(60, 256, device="cuda").bfloat16()
    made, freed, free = [], [], gf.Plan.free
    monkeypatch.setattr(gf.Plan, "free", lambda plan: (plan.handle and freed.append(plan.handle), free(plan)))
    init = gf.Plan.__init__
    monkeypatch.setattr(gf.Plan, "__init__", lambda plan, *args: (init(plan, *args), made.append(plan.handle))[0])
    first = [t.clone() for t in layer.train(x, x)]
    plans = len(made)
    second = layer.train(x, x)
    assert not freed and len(made) == plans  # the same choice: the same plans
    assert all(torch.equal(a, b) for a, b in zip(first, second))
