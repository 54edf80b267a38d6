"""The norm, the router and the activation's gradient at the most rows, tokens and
columns that their plans take (2^31 - 1, columns in eights)."""
import pytest
import torch

import gemm_epilogue_tmem_gb300 as gf

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1
PART = 2 ** 28


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    yield
    torch.cuda.empty_cache()


def _parts(n):
    return [slice(i, min(i + PART, n)) for i in range(0, n, PART)]


def _normal(n):
    gen = torch.Generator(device="cuda").manual_seed(1)
    out = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    for s in _parts(n):
        out[s] = torch.randn(s.stop - s.start, generator=gen, device="cuda")
    return out


def test_norm_of_the_most_rows():
    """hidden 1: y = w x / sqrt(x^2 + eps), d_x = w d eps (x^2 + eps)^-1.5; one rounding to bf16 (2^-8 of the
    value), and in fp32 a few steps of 2^-24 for y; the gradient is 1 - x^2 / (x^2 + eps), off by as many of 1 / sqrt."""
    eps = 0.5
    x, w = _normal(MOST), torch.tensor([1.5], dtype=torch.bfloat16, device="cuda")
    y, plan = torch.empty_like(x), gf.gf_rmsnorm_plan(MOST, 1, gf.GF_BF16, eps)
    gf.gf_rmsnorm_execute(plan, x, w, out=y)
    d_x, d_w = torch.empty_like(x), torch.empty(1, dtype=torch.float32, device="cuda")
    gf.gf_rmsnorm_grad_execute(plan, x, x, w, d_x, d_weight=d_w)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    total = 0.0
    for s in _parts(MOST):
        f = x[s].double()
        rstd = (f * f + eps).rsqrt()
        h = f * rstd
        want = 1.5 * h
        assert bool(((y[s].double() - want).abs() <= want.abs() * (2 ** -8 + 16 * 2 ** -24)).all())
        want = 1.5 * f * rstd * (1 - h * h)
        assert bool(((d_x[s].double() - want).abs() <= want.abs() * 2 ** -8 + 1.5 * h.abs() * 32 * 2 ** -24).all())
        total += float((f * h).sum())
    # fp32 sums of terms of one sign. A CTA has four thread rows here and every SM a CTA: at most 2^31 / (152 * 4) <
    # 2^21.8 terms a thread, each step off by 2^-24 of the sum so far, half the last on average: 2^-3 at worst
    assert abs(float(d_w) - total) <= total * 2 ** -3
    plan.free()


def test_router_of_the_most_tokens():
    x = _normal(MOST).view(MOST, 1)
    expert = torch.full((MOST, 1), -7, dtype=torch.int32, device="cuda")
    weight = torch.zeros(MOST, 1, device="cuda")
    plan = gf.gf_route_plan(MOST, 1, 1, gf.GF_BF16, gf.GF_SCORE_SIGMOID, renorm=False, scale=2.0)
    gf.gf_route_execute(plan, x, expert, weight)
    d_x = torch.empty_like(x)
    gf.gf_route_grad_execute(plan, x, expert, weight, d_x)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    for s in _parts(MOST):
        score = x[s].double().sigmoid()
        assert bool((expert[s] == 0).all())
        # the exponential, a sum, a division: a few steps of 2^-24
        assert bool(((weight[s].double() - 2 * score).abs() <= 2 * score * 16 * 2 ** -24).all())
        want = 4 * score * score * (1 - score)
        assert bool(((d_x[s].double() - want).abs() <= want * (2 ** -8 + 64 * 2 ** -24)).all())
    plan.free()


def test_gradient_of_the_most_columns():
    n = MOST // 8 * 8
    d, z = _normal(n).view(1, n), _normal(n).neg_().view(1, n)
    d_z, bgrad = torch.empty_like(d), torch.empty(n, dtype=torch.float32, device="cuda")
    plan = gf.gf_dact_bgrad_plan(1, n, gf.GF_BF16, gf.GF_ACT_RELU)
    gf.gf_dact_bgrad_execute(plan, d, z, d_z, bgrad)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    for s in _parts(n):
        want = torch.where(z[0, s] > 0, d[0, s].float(), torch.zeros((), device="cuda"))
        assert bool((d_z[0, s].float() == want).all()) and bool((bgrad[s] == want).all())
    plan.free()
