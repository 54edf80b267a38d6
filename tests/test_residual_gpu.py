"""out = act(A B + bias) + residual on the GPU, and the gradient of an activation and its bias, against the formulas in
64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_epilogue_tmem_gb300 as gf  # noqa: E402

TDT = {gf.GF_F16: torch.float16, gf.GF_BF16: torch.bfloat16}
# unit roundoff of the outputs, and the largest rounding error below the smallest normal
ROUND = {gf.GF_F16: (2.0 ** -11, 2.0 ** -25), gf.GF_BF16: (2.0 ** -8, 0.0)}
ACTS = [gf.GF_ACT_NONE, gf.GF_ACT_RELU, gf.GF_ACT_GELU, gf.GF_ACT_SILU]
C = math.sqrt(2 / math.pi)


def randn(*shape, seed, dtype, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (size * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def act(kind, z):
    if kind == gf.GF_ACT_RELU:
        return z.clamp(min=0)
    if kind == gf.GF_ACT_GELU:
        return 0.5 * z * (1 + torch.tanh(C * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z) if kind == gf.GF_ACT_SILU else z


def slope(kind, z):
    if kind == gf.GF_ACT_RELU:
        return (z > 0).double()
    if kind == gf.GF_ACT_SILU:
        s = torch.sigmoid(z)
        return s * (1 + z * torch.sigmoid(-z))
    t = torch.tanh(C * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * C * (1 + 3 * 0.044715 * z * z)


def filled(*shape, dtype):
    return torch.full(shape, float("nan"), device="cuda").to(dtype)


class Case:
    def __init__(self, m, n, k, dtype, layout, bias=True, seed=0):
        t = TDT[dtype]
        self.m, self.n, self.k, self.dtype, self.layout = m, n, k, dtype, layout
        self.a = randn(m, k, seed=seed, dtype=t)
        shape = (n, k) if layout == gf.GF_B_NK else (k, n)
        self.b = randn(*shape, seed=seed + 1, dtype=t, size=1 / math.sqrt(max(k, 1)))
        self.bias = randn(n, seed=seed + 2, dtype=t) if bias else None
        self.res = randn(m, n, seed=seed + 3, dtype=t)
        b = self.b.double()
        b = b.t() if layout == gf.GF_B_NK else b
        self.z = self.a.double() @ b
        # fp32 sums of k products in any order, and of the bias
        self.z_err = 2.0 ** -23 * (k + 1) * (self.a.double().abs() @ b.abs())
        if bias:
            self.z = self.z + self.bias.double()
            self.z_err = self.z_err + 2.0 ** -23 * self.z.abs()

    def run(self, plan, out=None, z_out=None, res=None):
        out = filled(self.m, self.n, dtype=TDT[self.dtype]) if out is None else out
        gf.gf_matmul_residual_execute(plan, self.a, self.b, self.res if res is None else res, out, bias=self.bias, z_out=z_out)
        assert gf.gf_plan_status(plan) == gf.GF_OK
        return out

    def check(self, kind, out, z=None):
        u, tiny = ROUND[self.dtype]
        a = act(kind, self.z)
        want = a + self.res.double()
        # slopes of the activations are below 1.13; exponential and division: 2^-20 of act(z)
        bound = want.abs() * (u + 2.0 ** -22) + 1.13 * self.z_err + 2.0 ** -19 * a.abs() + tiny
        err = (out.double() - want).abs()
        assert bool((err <= bound).all()), float((err - bound).max())
        if z is not None:
            assert bool(((z.double() - self.z).abs() <= self.z.abs() * u + self.z_err + tiny).all())


# m, n, k: single elements' worth; rows for each kernel; tails of every tile; nothing to multiply; long k
SHAPES = [(1, 8, 8), (1, 264, 1000), (3, 1024, 4096), (17, 200, 72), (16, 136, 512), (33, 4104, 264), (64, 72, 2056), (65, 520, 128), (130, 1000, 200),
          (257, 264, 1032), (1003, 2056, 520), (5, 64, 0), (300, 40, 8)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype,layout,kind,bias", [
    (gf.GF_F16, gf.GF_B_NK, gf.GF_ACT_GELU, True), (gf.GF_F16, gf.GF_B_KN, gf.GF_ACT_NONE, True),
    (gf.GF_BF16, gf.GF_B_NK, gf.GF_ACT_NONE, False), (gf.GF_BF16, gf.GF_B_KN, gf.GF_ACT_SILU, True),
    (gf.GF_BF16, gf.GF_B_KN, gf.GF_ACT_RELU, False)])
def test_forward(m, n, k, dtype, layout, kind, bias):
    c = Case(m, n, k, dtype, layout, bias)
    plan = gf.gf_matmul_residual_plan(m, n, k, dtype, kind, layout)
    z = filled(m, n, dtype=TDT[dtype])
    out = c.run(plan, z_out=z)
    c.check(kind, out, z)
    assert torch.equal(c.run(plan), out)  # z not kept
    inplace = c.res.clone()
    assert torch.equal(c.run(plan, out=inplace, res=inplace), out)  # into the residual
    plan.free()


@pytest.mark.parametrize("kernel,split", [(1, 0), (1, 3), (2, 0), (2, 3), (3, 0), (3, 2)])
@pytest.mark.parametrize("dtype,layout,kind", [(gf.GF_F16, gf.GF_B_NK, gf.GF_ACT_GELU), (gf.GF_BF16, gf.GF_B_KN, gf.GF_ACT_SILU)])
@pytest.mark.parametrize("m,n,k", [(300, 328, 520), (513, 1096, 1000), (2, 8, 136)])
def test_every_kernel(kernel, split, dtype, layout, kind, m, n, k):
    c = Case(m, n, k, dtype, layout, seed=40)
    plan = gf.gf_matmul_residual_plan(m, n, k, dtype, kind, layout)
    gf.gf_plan_set_option(plan, gf.GF_OPT_KERNEL, kernel)
    if split:
        gf.gf_plan_set_option(plan, gf.GF_OPT_SPLIT_K, split)
        assert gf.gf_plan_describe(plan)["k_splits"] == split
    z = filled(m, n, dtype=TDT[dtype])
    out = c.run(plan, z_out=z)
    c.check(kind, out, z)
    inplace = c.res.clone()
    assert torch.equal(c.run(plan, out=inplace, res=inplace), out)
    plan.free()


# rows of each tile height, and of several tiles; one k-block and many; tiles whole and dealt out; column tails with and
# without whole 64-column chunks
@pytest.mark.parametrize("m,n,k", [(1, 8, 8), (1, 5120, 1088), (7, 264, 4096), (16, 128, 64), (17, 200, 2056), (32, 1024, 520), (33, 72, 3000),
                                   (48, 4096, 1024), (64, 136, 8192), (65, 328, 1000), (128, 640, 2048), (129, 264, 520), (300, 72, 4104), (20, 64, 0),
                                   (5, 40000, 200), (1, 16, 65536)])
@pytest.mark.parametrize("dtype,layout,kind,bias", [(gf.GF_F16, gf.GF_B_NK, gf.GF_ACT_GELU, True), (gf.GF_BF16, gf.GF_B_KN, gf.GF_ACT_SILU, True),
                                                    (gf.GF_BF16, gf.GF_B_NK, gf.GF_ACT_NONE, False), (gf.GF_F16, gf.GF_B_KN, gf.GF_ACT_RELU, False)])
def test_few_rows(m, n, k, dtype, layout, kind, bias):
    c = Case(m, n, k, dtype, layout, bias, seed=50)
    plan = gf.gf_matmul_residual_plan(m, n, k, dtype, kind, layout)
    gf.gf_plan_set_option(plan, gf.GF_OPT_KERNEL, 4)
    z = filled(m, n, dtype=TDT[dtype])
    out = c.run(plan, z_out=z)
    c.check(kind, out, z)
    for _ in range(3):  # the same bits whichever CTA ends last, and into the residual
        inplace = c.res.clone()
        assert torch.equal(c.run(plan, out=inplace, res=inplace), out)
    plan.free()


def test_few_rows_times_out_and_recovers():
    """A load that never comes: the waits run out, the status says so, and the plan works again."""
    c = Case(3, 256, 4096, gf.GF_BF16, gf.GF_B_NK, seed=55)
    plan = gf.gf_matmul_residual_plan(3, 256, 4096, gf.GF_BF16, gf.GF_ACT_NONE, gf.GF_B_NK)
    gf.gf_plan_set_option(plan, gf.GF_OPT_WAIT_LIMIT_US, 20000)
    gf.gf_plan_set_option(plan, gf.GF_OPT_FAULT_DROP_LOAD, 2)
    out = torch.empty_like(c.res)
    gf.gf_matmul_residual_execute(plan, c.a, c.b, c.res, out, bias=c.bias)
    assert gf.gf_plan_status(plan) == gf.GF_ERR_DEVICE_TIMEOUT
    gf.gf_plan_set_option(plan, gf.GF_OPT_FAULT_DROP_LOAD, 0)
    c.check(gf.GF_ACT_NONE, c.run(plan))
    plan.free()


def test_without_an_activation_it_is_the_product_and_the_sum():
    """The same kernel without a bias and with a residual of zeros gives the bits of the plain product."""
    c = Case(300, 328, 520, gf.GF_BF16, gf.GF_B_NK, bias=False, seed=60)
    c.res.zero_()
    plain = gf.gf_matmul_plan_ex(300, 328, 520, gf.GF_BF16, gf.GF_EPILOG_NONE, gf.GF_BIAS_COL, gf.GF_B_NK)
    want = torch.empty_like(c.res)
    gf.gf_matmul_execute(plain, c.a, c.b, out=want)
    plan = gf.gf_matmul_residual_plan(300, 328, 520, gf.GF_BF16, gf.GF_ACT_NONE, gf.GF_B_NK)
    for kernel in (1, 2, 3):
        gf.gf_plan_set_option(plain, gf.GF_OPT_KERNEL, kernel)
        gf.gf_plan_set_option(plan, gf.GF_OPT_KERNEL, kernel)
        gf.gf_matmul_execute(plain, c.a, c.b, out=want)
        assert torch.equal(c.run(plan), want)
    plain.free()
    plan.free()


@pytest.mark.parametrize("m,n", [(0, 8), (1, 8), (7, 256), (33, 264), (1000, 72), (513, 2056), (4100, 520)])
@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("dtype", [gf.GF_F16, gf.GF_BF16])
def test_dact_bgrad(m, n, kind, dtype):
    t, (u, tiny) = TDT[dtype], ROUND[dtype]
    dy, z = randn(m, n, seed=70, dtype=t), randn(m, n, seed=71, dtype=t, size=3.0)
    if m > 6:
        z[0], z[1], z[2, ::2] = 0, float("inf"), -30.0
    plan = gf.gf_dact_bgrad_plan(m, n, dtype, kind)
    bgrad = filled(n, dtype=torch.float32)
    if kind == gf.GF_ACT_NONE:
        gf.gf_dact_bgrad_execute(plan, dy, bgrad=bgrad)
        d = dy.double()
        err = torch.zeros_like(d)
    else:
        d_z = filled(m, n, dtype=t)
        gf.gf_dact_bgrad_execute(plan, dy, z=z, d_z=d_z, bgrad=bgrad)
        zd = z.double().clamp(max=100.0)  # the slope's limit
        d = dy.double() * slope(kind, zd)
        # the logistic's error, 2^-21, times z u'(z), which is below 2^6 where the logistic's slope is above 2^-24
        err = (0.0 if kind == gf.GF_ACT_RELU else 2.0 ** -16) * dy.double().abs()
        assert bool(((d_z.double() - d).abs() <= d.abs() * u + err + tiny).all())
        again, b2 = dy.clone(), torch.empty_like(bgrad)
        gf.gf_dact_bgrad_execute(plan, again, z=z, d_z=again, bgrad=b2)  # in place
        assert torch.equal(again, d_z) and torch.equal(b2, bgrad)
        gf.gf_dact_bgrad_execute(plan, dy, z=z, d_z=again)
        assert torch.equal(again, d_z)
    bound = 2.0 ** -24 * (m + 64) * d.abs().sum(0) + err.sum(0)
    assert bool(((bgrad.double() - d.sum(0)).abs() <= bound).all())
    plan.free()


def test_refusals():
    for args, status in (((8, 12, 8, gf.GF_F16, 0, 0), gf.GF_ERR_UNSUPPORTED), ((8, 8, 8, gf.GF_F16, 4, 0), gf.GF_ERR_INVALID_VALUE),
                         ((8, 8, 8, gf.GF_F32, 0, 0), gf.GF_ERR_INVALID_VALUE)):
        with pytest.raises(gf.GfError) as e:
            gf.gf_matmul_residual_plan(*args)
        assert e.value.status == status
    c = Case(16, 64, 32, gf.GF_BF16, gf.GF_B_KN)
    plan = gf.gf_matmul_residual_plan(16, 64, 32, gf.GF_BF16)
    out = torch.empty_like(c.res)
    for call in (lambda: gf.gf_matmul_residual_execute(plan, c.a, c.b, None, out),
                 lambda: gf.gf_matmul_residual_execute(plan, c.a, c.b, c.res, None),
                 lambda: gf.gf_matmul_residual_execute(plan, c.a, c.b, c.res.half(), out),
                 lambda: gf.gf_matmul_residual_execute(plan, c.a, c.b, c.res, out, bias=c.bias[:8]),
                 lambda: gf.gf_matmul_residual_execute(plan, c.a, c.b, c.res.data_ptr() + 2, out),
                 lambda: gf.gf_matmul_residual_execute(plan, c.a, c.b, c.res, out, bias=c.bias.data_ptr() + 2),
                 lambda: gf.gf_matmul_residual_execute(plan, c.a, c.b, c.res, out, z_out=out.data_ptr() + 2),
                 lambda: gf.gf_matmul_execute(plan, c.a, c.b, out=out),  # another plan's call
                 lambda: gf.gf_matmul_autotune(plan, c.a, c.b, out=out)):
        with pytest.raises(gf.GfError):
            call()
    plan.free()
    plan = gf.gf_dact_bgrad_plan(16, 64, gf.GF_BF16, gf.GF_ACT_GELU)
    bg = torch.empty(64, device="cuda")
    for call in (lambda: gf.gf_dact_bgrad_execute(plan, c.res, z=c.res, bgrad=bg), lambda: gf.gf_dact_bgrad_execute(plan, c.res, d_z=out),
                 lambda: gf.gf_dact_bgrad_execute(plan, c.res, z=c.res, d_z=out, bgrad=bg.half())):
        with pytest.raises(gf.GfError):
            call()
    plan.free()
    plan = gf.gf_dact_bgrad_plan(16, 64, gf.GF_BF16, gf.GF_ACT_NONE)
    for call in (lambda: gf.gf_dact_bgrad_execute(plan, c.res), lambda: gf.gf_dact_bgrad_execute(plan, c.res, z=c.res, d_z=out, bgrad=bg)):
        with pytest.raises(gf.GfError):
            call()
    plan.free()
