"""A plan's device words (counters, status) are set before any stream can use them."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

AT_ONCE_ON_A_SIDE_STREAM = """
import sys
import torch
import gemm_epilogue_tmem_gb300 as gf
gen = torch.Generator(device="cuda").manual_seed(1)
if sys.argv[1] == "e4m3":
    m, n, k = 1, 4096, 8192  # 32 tiles, each split over several CTAs
    a = torch.randn(m, k, generator=gen, device="cuda").to(torch.float8_e4m3fn)
    b = torch.randn(1, n, k, generator=gen, device="cuda").to(torch.float8_e4m3fn)
    sa, sb = torch.ones(m, k // 128, device="cuda"), torch.ones(1, n // 128, k // 128, device="cuda")

    def make():
        return gf.gf_fp8_matmul_plan(m, n, k, 1, gf.GF_BF16)

    def run(plan, out, **stream):
        gf.gf_fp8_matmul_execute(plan, a, sa, b, sb, out=out, **stream)
else:
    m, n, k = 256, 512, 2048  # 8 tiles, k split
    a = torch.randn(m, k, generator=gen, device="cuda").bfloat16()
    b = torch.randn(k, n, generator=gen, device="cuda").bfloat16()

    def make():
        plan = gf.gf_matmul_plan(m, n, k, gf.GF_BF16, gf.GF_EPILOG_NONE)
        assert gf.gf_plan_describe(plan)["k_splits"] > 1
        return plan

    def run(plan, out, **stream):
        gf.gf_matmul_execute(plan, a, b, out=out, **stream)

calls = 300
out = torch.empty(calls, m, n, dtype=torch.bfloat16, device="cuda")
plan = make()
run(plan, out[0])
torch.cuda.synchronize()
want = out[0].clone()
plan.free()
side = torch.cuda.Stream()
wrong = 0
for turn in range(40):
    out.fill_(7)
    torch.cuda.synchronize()
    torch.cuda._sleep(2_000_000 + 10_000 * turn)  # 1 ms of the default stream, over while the products run
    plan = make()
    for i in range(calls):
        run(plan, out[i], stream=side)
    side.synchronize()
    assert gf.gf_plan_status(plan, stream=side) == gf.GF_OK
    wrong += int((out != want).any(dim=2).any(dim=1).sum())
    plan.free()
print("wrong", wrong)
"""


@pytest.mark.parametrize("product", ["e4m3", "bf16"])
def test_first_call_on_another_stream(product):
    """A plan made while the default stream is busy, executed at once on a stream that does not wait for it: nothing of
    the plan's creation may still be to come, such as the zeroing of the counters by which the parts of a tile join."""
    r = subprocess.run([sys.executable, "-c", AT_ONCE_ON_A_SIDE_STREAM, product], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "wrong 0", r.stdout[-500:] + r.stderr[-2000:]
