"""The norm, the router and the products with a residual without a GPU: plans and calls reject invalid arguments before
touching a device; the router's reference against hand-worked rows; the sources' rules."""
import os
import re

import numpy as np
import pytest

import gemm_epilogue_tmem_gb300 as gf
from route_reference import route, route_grad, scores

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_epilogue_tmem_gb300", "csrc")
INVALID, UNSUPPORTED = gf.GF_ERR_INVALID_VALUE, gf.GF_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    gf.build()
    return gf.lib()


GOOD = (8, 16, 2, 2, 1, 1, 1.0, 4, 2, 2, 16)  # tokens, experts, topk, dtype, score, renorm, scale, groups, topk_groups, best, ld


@pytest.mark.parametrize("at,value,status", [
    (0, -1, INVALID), (0, 1 << 30, INVALID), (1, 0, INVALID), (1, 1025, INVALID), (2, 0, INVALID), (2, 65, INVALID), (2, 9, INVALID), (3, 3, INVALID),
    (4, 2, INVALID), (5, 2, INVALID), (6, float("inf"), INVALID), (6, float("nan"), INVALID), (7, 0, INVALID), (7, 3, INVALID), (7, 17, INVALID),
    (8, 0, INVALID), (8, 5, INVALID), (9, 0, INVALID), (9, 3, INVALID), (10, 15, INVALID), (10, (1 << 24) + 1, INVALID)])
def test_route_plan_rejects_before_device(L, at, value, status):
    args = list(GOOD)
    args[at] = value
    assert not L.gf_route_plan(*args)
    assert L.gf_last_error() == status


def test_too_many_groups(L):
    assert not L.gf_route_plan(8, 66, 2, 2, 1, 1, 1.0, 33, 2, 2, 66)
    assert L.gf_last_error() == UNSUPPORTED


@pytest.mark.parametrize("args,status", [
    ((-1, 64, 0, 1e-6), INVALID), ((4, 0, 0, 1e-6), INVALID), ((4, 64, 2, 1e-6), INVALID), ((4, 64, 0, -1.0), INVALID),
    ((4, 64, 0, float("nan")), INVALID), ((4, 64, 0, float("inf")), INVALID), ((4, 32769, 0, 1e-6), UNSUPPORTED), ((1 << 31, 64, 0, 1e-6), INVALID)])
def test_rmsnorm_plan_rejects_before_device(L, args, status):
    assert not L.gf_rmsnorm_plan(*args)
    assert L.gf_last_error() == status


@pytest.mark.parametrize("args,status", [
    ((-1, 8, 8, 0, 0, 0), INVALID), ((8, 8, 8, 2, 0, 0), INVALID), ((8, 8, 8, 0, 4, 0), INVALID), ((8, 8, 8, 0, -1, 0), INVALID),
    ((8, 8, 8, 0, 0, 2), INVALID), ((8, 12, 8, 0, 0, 0), UNSUPPORTED), ((8, 8, 12, 0, 0, 0), UNSUPPORTED)])
def test_residual_plan_rejects_before_device(L, args, status):
    assert not L.gf_matmul_residual_plan(*args)
    assert L.gf_last_error() == status


@pytest.mark.parametrize("args,status", [
    ((-1, 8, 0, 0), INVALID), ((8, -8, 0, 0), INVALID), ((8, 8, 2, 0), INVALID), ((8, 8, 0, 4), INVALID), ((8, 12, 0, 0), UNSUPPORTED),
    ((1 << 31, 8, 0, 0), INVALID)])
def test_dact_plan_rejects_before_device(L, args, status):
    assert not L.gf_dact_bgrad_plan(*args)
    assert L.gf_last_error() == status


def test_null_plans(L):
    assert L.gf_route_execute(*[None] * 6) == INVALID
    assert L.gf_route_grad_execute(*[None] * 6) == INVALID
    assert L.gf_rmsnorm_execute(*[None] * 9) == INVALID
    assert L.gf_rmsnorm_grad_execute(*[None] * 8) == INVALID
    assert L.gf_matmul_residual_execute(*[None] * 8) == INVALID
    assert L.gf_dact_bgrad_execute(*[None] * 6) == INVALID


def test_no_device_here(L):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for plan in (L.gf_route_plan(*GOOD), L.gf_rmsnorm_plan(4, 64, 0, 1e-6), L.gf_matmul_residual_plan(8, 8, 8, 0, 0, 0), L.gf_dact_bgrad_plan(8, 8, 0, 0)):
        assert not plan and L.gf_last_error() == gf.GF_ERR_NO_DEVICE


@pytest.mark.parametrize("name", ["k_route.cu", "two_float.cuh", "k_norm.cu", "norm_common.cuh", "k_norm_stream.cu", "k_dact.cu", "k_residual_narrow.cu"])
def test_no_read_only_loads(name):
    """Launched while the kernel that writes their inputs may still run, and some in place: no loads that take data for constant."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in code, word


def test_reference_by_hand():
    l = np.array([[1.0, 3.0, 3.0, 0.0, 2.0, -np.inf]])
    e, w = route(l, 3, False, True, 2.0)
    assert e.tolist() == [[1, 2, 4]]  # ties to the lowest index
    p = np.exp([3.0, 3.0, 2.0])
    assert np.allclose(w, 2 * p / p.sum())
    # groups of two: sums of scores 4, 3 + s, 2; the best two stay
    e, _ = route(l, 3, False, True, 1.0, None, 3, 1, 1)
    assert e.tolist() == [[1, 0, -1]]
    # a bias that only the choice sees
    e, w = route(l, 2, True, False, 1.0, np.array([0, 0, 0, 5.0, 0, 9.0]))
    assert e.tolist() == [[3, 1]] and np.allclose(w, scores(l, True)[0, [3, 1]])


def test_reference_gradient_by_differences():
    rng = np.random.default_rng(0)
    l, g = rng.standard_normal((1, 9)), rng.standard_normal((1, 3))
    for sigmoid in (True, False):
        for renorm in (True, False):
            e, _ = route(l, 3, sigmoid, renorm, 1.3)
            d, _ = route_grad(l, e, g, sigmoid, renorm, 1.3)
            for j in range(9):
                h = np.zeros_like(l)
                h[0, j] = 1e-6
                up, down = (route(l + s * h, 3, sigmoid, renorm, 1.3)[1] for s in (1, -1))
                assert abs(((up - down) * g).sum() / 2e-6 - d[0, j]) < 1e-7
