"""Expert routing and the e4m3 operators without a GPU: their plans and calls
reject invalid arguments before touching a device; the quantiser's reference
against torch's e4m3 conversion."""
import numpy as np
import pytest

import gemm_epilogue_tmem_gb300 as gf
from fp8_reference import block_scale, dequantize, quantize_reference, round_e4m3


@pytest.fixture(scope="module")
def L():
    gf.build()
    return gf.lib()


@pytest.mark.parametrize("args,status", [
    ((-1, 2, 4, 64, 0), gf.GF_ERR_INVALID_VALUE),
    ((8, 0, 4, 64, 0), gf.GF_ERR_INVALID_VALUE),
    ((8, 65, 100, 64, 0), gf.GF_ERR_INVALID_VALUE),
    ((8, 2, 0, 64, 0), gf.GF_ERR_INVALID_VALUE),
    ((8, 2, 1025, 64, 0), gf.GF_ERR_INVALID_VALUE),
    ((8, 2, 4, 0, 0), gf.GF_ERR_INVALID_VALUE),
    ((8, 2, 4, (1 << 24) + 1, 0), gf.GF_ERR_INVALID_VALUE),
    ((8, 2, 4, 64, 2), gf.GF_ERR_INVALID_VALUE),
    ((1 << 30, 2, 4, 64, 0), gf.GF_ERR_INVALID_VALUE),   # tokens * topk >= 2^31
])
def test_moe_plan_rejects_before_device(L, args, status):
    assert not L.gf_moe_plan(*args)
    assert L.gf_last_error() == status


@pytest.mark.parametrize("args,status", [
    ((-1, 128, 128, 1, 0, 0), gf.GF_ERR_INVALID_VALUE),
    ((8, 128, 128, 0, 0, 0), gf.GF_ERR_INVALID_VALUE),
    ((8, 128, 128, 1025, 0, 0), gf.GF_ERR_INVALID_VALUE),
    ((8, 128, 128, 1, 3, 0), gf.GF_ERR_INVALID_VALUE),
    ((8, 128, 128, 1, 0, 2), gf.GF_ERR_INVALID_VALUE),
    ((8, 128, 24, 1, 0, 0), gf.GF_ERR_UNSUPPORTED),      # k % 16
    ((8, 12, 128, 1, 0, 0), gf.GF_ERR_UNSUPPORTED),      # n % 8
    ((8, 24, 128, 1, 0, 1), gf.GF_ERR_UNSUPPORTED),      # n % 16 for the e4m3 output
    ((8, 1 << 22, 128, 1024, 0, 0), gf.GF_ERR_UNSUPPORTED),  # groups * n
    ((1 << 31, 128, 128, 1, 0, 0), gf.GF_ERR_INVALID_VALUE),
    (((1 << 31) - 512, 128, 16, 1, 0, 0), gf.GF_ERR_UNSUPPORTED),     # rows past the last tile
    ((1 << 24, 1 << 20, 16, 1, 0, 0), gf.GF_ERR_UNSUPPORTED),         # tiles
])
def test_fp8_plan_rejects_before_device(L, args, status):
    assert not L.gf_fp8_matmul_plan(*args)
    assert L.gf_last_error() == status


@pytest.mark.parametrize("args,status", [
    ((-1, 128, 0, 1, None, None, None, None), gf.GF_ERR_INVALID_VALUE),
    ((4, 128, 2, 1, None, None, None, None), gf.GF_ERR_INVALID_VALUE),
    ((4, 128, 0, 64, None, None, None, None), gf.GF_ERR_INVALID_VALUE),
    ((4, 120, 0, 1, None, None, None, None), gf.GF_ERR_UNSUPPORTED),
    ((4, 128, 0, 1, None, None, None, None), gf.GF_ERR_INVALID_VALUE),   # no pointers
    ((4, 128, 0, 1, 16, 17, 16, None), gf.GF_ERR_INVALID_VALUE),         # misaligned
])
def test_quantize_rejects_before_device(L, args, status):
    assert L.gf_fp8_quantize(*args) == status
    assert L.gf_last_error() == status


def test_null_plans(L):
    assert L.gf_moe_dispatch_execute(*[None] * 8) == gf.GF_ERR_INVALID_VALUE
    assert L.gf_moe_dispatch_fp8_execute(*[None] * 9) == gf.GF_ERR_INVALID_VALUE
    assert L.gf_moe_dispatch_grad_execute(*[None] * 5) == gf.GF_ERR_INVALID_VALUE
    assert L.gf_moe_combine_execute(*[None] * 6) == gf.GF_ERR_INVALID_VALUE
    assert L.gf_moe_combine_grad_execute(*[None] * 9) == gf.GF_ERR_INVALID_VALUE
    assert L.gf_fp8_matmul_execute(*[None] * 11) == gf.GF_ERR_INVALID_VALUE


def test_no_device_here(L):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert not L.gf_moe_plan(8, 2, 4, 64, 0) and L.gf_last_error() == gf.GF_ERR_NO_DEVICE
    assert not L.gf_fp8_matmul_plan(8, 128, 128, 1, 0, 0)
    assert L.gf_last_error() == gf.GF_ERR_NO_DEVICE


def test_rounding_against_torch():
    torch = pytest.importorskip("torch")
    v = torch.cat([torch.linspace(-448, 448, 20011), torch.arange(-64, 65) / 1024.0])
    v = torch.cat([v, torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()])
    v = v[v.isfinite()]
    want = v.to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(round_e4m3(v.double().numpy()), want)


def test_scale_is_the_smallest_power_of_two():
    for amax in (448.0, 448.25, 447.75, 1e-40, 3e38, 0.4375, 1.0, 2.0 ** -126 * 448):
        s = block_scale(amax)
        assert amax / s <= 448 and (s == 2.0 ** -126 or amax / (s / 2) > 448)
    assert block_scale(0.0) == 1.0
    x = np.random.default_rng(0).standard_normal((300, 272))
    for rows in (1, 128):
        q, s = quantize_reference(x, rows)
        assert np.abs(q).max() <= 448
        assert np.abs(dequantize(q, s, rows) - x).max() <= 2.0 ** -4 * np.abs(x).max()
