"""Root-mean-square norm on the GPU, forward (16 bits, e4m3) and backward, against the formulas in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_epilogue_tmem_gb300 as gf  # noqa: E402

TDT = {gf.GF_F16: torch.float16, gf.GF_BF16: torch.bfloat16}
# unit roundoff of the outputs, and the largest rounding error below the smallest normal
ROUND = {gf.GF_F16: (2.0 ** -11, 2.0 ** -25), gf.GF_BF16: (2.0 ** -8, 0.0)}
EPS = 1e-5

# rows, hidden: one element; rows that begin anywhere in a 16-byte word and lie within one; several rows a CTA, one and
# more words a thread; the longest, whole and odd
SHAPES = [(1, 1), (3, 5), (9, 8), (70, 16), (33, 17), (257, 130), (40, 1000), (5, 1027), (700, 2047), (3, 2048), (17, 4095),
          (2, 5120), (19, 8190), (3, 8192), (2, 16385), (3, 20000), (2, 32767), (2, 32768)]

# many rows of whole words, which stream through shared memory: short ones that share a turn, a last turn that is not
# full, one and more words a thread, rows of which a ring holds two
MANY = [(40001, 8), (9005, 64), (7003, 1024), (4099, 136), (1000, 2048), (1500, 5120), (701, 8192), (400, 16384), (320, 20000), (310, 32768)]


def randn(*shape, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def inputs(rows, hidden, dtype, seed=1):
    t = TDT[dtype]
    size = torch.exp(torch.linspace(-3, 3, rows, device="cuda"))[:, None]
    x = (randn(rows, hidden, seed=seed, dtype=torch.float32) * size).to(t)
    return x, randn(rows, hidden, seed=seed + 1, dtype=t), (1 + 0.3 * randn(hidden, seed=seed + 2, dtype=torch.float32)).to(t)


def exact(r, w):
    r = r.double()
    inv = (r.square().mean(1, keepdim=True) + EPS) ** -0.5
    return r * inv * w.double(), inv


def near(got, want, dtype, extra=0.0):
    """Within one rounding of `want`, plus `extra` absolute and fp32's errors: sums of at most 80 terms in a row."""
    u, tiny = ROUND[dtype]
    err = (got.double() - want).abs()
    bound = want.abs() * (u + 2.0 ** -17) + tiny + extra
    assert bool((err <= bound).all()), float((err - bound).max())


def filled(*shape, dtype):
    return torch.full(shape, float("nan"), device="cuda").to(dtype)


@pytest.mark.parametrize("rows,hidden", SHAPES + MANY)
@pytest.mark.parametrize("dtype", [gf.GF_F16, gf.GF_BF16])
def test_forward(rows, hidden, dtype):
    t = TDT[dtype]
    x, res, w = inputs(rows, hidden, dtype)
    plan = gf.gf_rmsnorm_plan(rows, hidden, dtype, EPS)
    out, r_out = filled(rows, hidden, dtype=t), filled(rows, hidden, dtype=t)
    gf.gf_rmsnorm_execute(plan, x, w, out=out)
    near(out, exact(x, w)[0], dtype)
    gf.gf_rmsnorm_execute(plan, x, w, residual=res, residual_out=r_out, out=out)
    r = (x.float() + res.float()).to(t)
    assert torch.equal(r_out, r)
    near(out, exact(r, w)[0], dtype)
    # the sum not kept; the sum and the norm in place of the inputs
    again = filled(rows, hidden, dtype=t)
    gf.gf_rmsnorm_execute(plan, x, w, residual=res, out=again)
    assert torch.equal(again, out)
    a, b = x.clone(), res.clone()
    gf.gf_rmsnorm_execute(plan, a, w, residual=b, residual_out=b, out=a)
    assert torch.equal(a, out) and torch.equal(b, r)
    plan.free()


@pytest.mark.parametrize("rows,hidden", [(1, 16), (5, 128), (3, 144), (66, 1040), (1, 5120), (31, 8192), (2, 16400), (3, 32768)] +
                         [(rows, hidden) for rows, hidden in MANY if hidden % 16 == 0])
@pytest.mark.parametrize("dtype", [gf.GF_F16, gf.GF_BF16])
def test_e4m3(rows, hidden, dtype):
    t, blocks = TDT[dtype], -(-hidden // 128)
    x, res, w = inputs(rows, hidden, dtype, seed=5)
    if rows > 2:
        x[1] = 0
        res[1] = 0  # a row of zeros
        w[:min(hidden, 128)] = 0  # a block of zeros
    plan = gf.gf_rmsnorm_plan(rows, hidden, dtype, EPS)
    q = torch.full((rows, hidden), 0x55, dtype=torch.uint8, device="cuda")
    scale, out, r_out = filled(rows, blocks, dtype=torch.float32), filled(rows, hidden, dtype=t), filled(rows, hidden, dtype=t)
    gf.gf_rmsnorm_execute(plan, x, w, residual=res, residual_out=r_out, out=out, out8=q, out_scale=scale)
    r = (x.float() + res.float()).to(t)
    y = exact(r, w)[0]
    assert torch.equal(r_out, r)
    near(out, y, dtype)
    pad = torch.nn.functional.pad(y, (0, -hidden % 128)).view(rows, blocks, 128)
    top = pad.abs().amax(2)
    power = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), 0.0)
    power = torch.where((top > 0) & (torch.exp2(power - 1) * 448 >= top), power - 1, power)
    want = torch.exp2(power.clamp(min=-126))
    assert torch.equal(scale.double(), want)
    v = y / want.repeat_interleave(128, 1)[:, :hidden]
    got = q.view(torch.float8_e4m3fn).double()
    bound = torch.maximum(v.abs() * (2.0 ** -4 + 2.0 ** -17), torch.full_like(v, 2.0 ** -10 * (1 + 2.0 ** -17)))
    assert bool(((got - v).abs() <= bound).all())
    # alone, and a scale that is a part of a larger array
    q2, part = torch.empty_like(q), torch.empty(rows * blocks + 1, device="cuda")[1:]
    gf.gf_rmsnorm_execute(plan, x, w, residual=res, out8=q2, out_scale=part)
    assert torch.equal(q, q2) and torch.equal(part.view(rows, blocks), scale)
    plan.free()


@pytest.mark.parametrize("rows", [250, 8192])  # loaded by their CTA, and streamed
def test_scales_at_the_border(rows):
    """Blocks whose largest value is 448 times a power of two, and as near to it as inputs allow: the scale of 64 bits."""
    hidden = 256
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, hidden, generator=g, device="cuda").half()
    w = torch.ones(hidden, device="cuda").half()
    # a weight for one column that brings this row's y there next to 1.75: rows with a sum of squares near each other
    x[:, 7] = 1.75
    want_ms = 1.0
    for _ in range(40):  # scale the others until the mean square is 1 up to fp16's steps
        ms = x.double().square().sum(1) - 1.75 ** 2
        f = ((want_ms * hidden - 1.75 ** 2) / ms).sqrt()
        new = (x.double() * f[:, None]).half()
        new[:, 7] = 1.75
        x = new
    plan = gf.gf_rmsnorm_plan(rows, hidden, gf.GF_F16, 0.0)
    q, scale = torch.empty(rows, hidden, dtype=torch.uint8, device="cuda"), torch.empty(rows, 2, device="cuda")
    w[:128] = 2.0 ** -3
    w[7] = 1  # the block's largest by far
    gf.gf_rmsnorm_execute(plan, x, w, out8=q, out_scale=scale)
    y = x.double() * w.double() / x.double().square().mean(1, keepdim=True).sqrt()
    top = y[:, :128].abs().amax(1)
    assert int(((top / 1.75 - 1).abs() < 1e-4).sum()) > rows // 4  # the case is what it says
    want = torch.where(top > 1.75, 2.0 ** -7, 2.0 ** -8)
    assert torch.equal(scale[:, 0].double(), want)
    plan.free()


@pytest.mark.parametrize("rows", [6, 6000])
def test_values_without_a_number(rows):
    hidden = 256
    x, _, w = inputs(rows, hidden, gf.GF_BF16)
    x[1, 3] = float("nan")
    x[2, 200] = float("inf")
    plan = gf.gf_rmsnorm_plan(rows, hidden, gf.GF_BF16, EPS)
    out, q = torch.empty_like(x), torch.empty(rows, hidden, dtype=torch.uint8, device="cuda")
    scale = torch.empty(rows, 2, device="cuda")
    gf.gf_rmsnorm_execute(plan, x, w, out=out, out8=q, out_scale=scale)
    v = q.view(torch.float8_e4m3fn).float()
    for got in (out.float(), v):
        assert bool(got[1].isnan().all())
        assert bool(got[2, 200].isnan()) and bool((got[2, :128] == 0).all())
        assert bool(got[[0, 3, 4, 5]].isfinite().all())
    assert bool((scale[1:3] == 1).all())
    plan.free()


@pytest.mark.parametrize("rows,hidden", SHAPES + MANY + [(5003, 136), (4099, 250), (999, 1027)])
@pytest.mark.parametrize("dtype,along", [(gf.GF_F16, True), (gf.GF_BF16, True), (gf.GF_BF16, False)])
def test_backward(rows, hidden, dtype, along):
    t = TDT[dtype]
    r, d_res, w = inputs(rows, hidden, dtype, seed=11)
    dy = randn(rows, hidden, seed=20, dtype=t)
    plan = gf.gf_rmsnorm_plan(rows, hidden, dtype, EPS)
    d_x, d_w = filled(rows, hidden, dtype=t), filled(hidden, dtype=torch.float32)
    res = d_res if along else None
    gf.gf_rmsnorm_grad_execute(plan, dy, r, w, d_x, d_weight=d_w, d_residual=res)
    _, inv = exact(r, w)
    h, g = r.double() * inv, dy.double() * w.double()
    mean, most = (g * h).mean(1, keepdim=True), (g * h).abs().mean(1, keepdim=True)
    want = inv * (g - h * mean)
    extra = 2.0 ** -16 * inv * (g.abs() + h.abs() * most)
    if along:
        want = want + d_res.double()
    near(d_x, want, dtype, extra)
    terms = dy.double() * h
    bound = (2.0 ** -24 * (rows + 100) + 2.0 ** -17) * terms.abs().sum(0)
    assert bool(((d_w.double() - terms.sum(0)).abs() <= bound).all())
    # the same bits again, in place, and without the weight's
    again, w2 = dy.clone(), filled(hidden, dtype=torch.float32)
    gf.gf_rmsnorm_grad_execute(plan, again, r, w, again, d_weight=w2, d_residual=res)
    assert torch.equal(again, d_x) and torch.equal(w2, d_w)
    if along:
        again = d_res.clone()
        gf.gf_rmsnorm_grad_execute(plan, dy, r, w, again, d_residual=again)
        assert torch.equal(again, d_x)
    plan.free()


def test_backward_against_differences():
    rows, hidden = 3, 24
    x, _, w = inputs(rows, hidden, gf.GF_F16, seed=30)
    dy = randn(rows, hidden, seed=31, dtype=torch.float16)
    plan = gf.gf_rmsnorm_plan(rows, hidden, gf.GF_F16, EPS)
    d_x, d_w = torch.empty_like(x), torch.empty(hidden, device="cuda")
    gf.gf_rmsnorm_grad_execute(plan, dy, x, w, d_x, d_weight=d_w)
    step, xd, wd = 1e-5, x.double(), w.double()

    def loss(a, b):
        return float((a / (a.square().mean(1, keepdim=True) + EPS).sqrt() * b * dy.double()).sum())

    for i, j in [(0, 0), (1, 7), (2, 23)]:
        d = torch.zeros_like(xd)
        d[i, j] = step
        slope = (loss(xd + d, wd) - loss(xd - d, wd)) / (2 * step)
        assert abs(slope - float(d_x[i, j])) <= 2.0 ** -10 * abs(slope) + 1e-5
        slope = (loss(xd, wd + d[i]) - loss(xd, wd - d[i])) / (2 * step)
        assert abs(slope - float(d_w[j])) <= 1e-5 * abs(slope) + 1e-5
    plan.free()


def test_times_out_and_recovers():
    """A copy that is never asked for: the waits run out, the status says so, and the plan works again."""
    rows, hidden = 4000, 1024
    x, res, w = inputs(rows, hidden, gf.GF_BF16)
    plan = gf.gf_rmsnorm_plan(rows, hidden, gf.GF_BF16, EPS)
    gf.gf_plan_set_option(plan, gf.GF_OPT_WAIT_LIMIT_US, 20000)
    gf.gf_plan_set_option(plan, gf.GF_OPT_FAULT_DROP_LOAD, 2)
    out, d_w = torch.empty_like(x), torch.empty(hidden, device="cuda")
    for call in (lambda: gf.gf_rmsnorm_execute(plan, x, w, residual=res, out=out), lambda: gf.gf_rmsnorm_grad_execute(plan, res, x, w, out, d_weight=d_w)):
        call()
        assert gf.gf_plan_status(plan) == gf.GF_ERR_DEVICE_TIMEOUT
        assert gf.gf_plan_status(plan) == gf.GF_OK
    gf.gf_plan_set_option(plan, gf.GF_OPT_FAULT_DROP_LOAD, 0)
    gf.gf_rmsnorm_execute(plan, x, w, out=out)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    near(out, exact(x, w)[0], gf.GF_BF16)
    plan.free()


def test_no_rows():
    plan = gf.gf_rmsnorm_plan(0, 64, gf.GF_BF16)
    none = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    d_w = torch.full((64,), float("nan"), device="cuda")
    gf.gf_rmsnorm_execute(plan, none, w, out=none)
    gf.gf_rmsnorm_grad_execute(plan, none, none, w, none, d_weight=d_w)
    assert bool((d_w == 0).all())
    plan.free()


def test_refusals():
    with pytest.raises(gf.GfError):
        gf.gf_rmsnorm_plan(4, 32769, gf.GF_BF16)
    plan = gf.gf_rmsnorm_plan(4, 72, gf.GF_BF16)
    x = torch.zeros(4, 72, dtype=torch.bfloat16, device="cuda")
    w, s = x[0].clone(), torch.zeros(4, 1, device="cuda")
    q = torch.zeros(4, 72, dtype=torch.uint8, device="cuda")
    for call in (lambda: gf.gf_rmsnorm_execute(plan, x, w),                                   # no output
                 lambda: gf.gf_rmsnorm_execute(plan, x, w, out8=q, out_scale=s),              # hidden % 16
                 lambda: gf.gf_rmsnorm_execute(plan, x, w, out=x, out8=q),                    # no scale
                 lambda: gf.gf_rmsnorm_execute(plan, x, w, residual_out=x, out=x),            # nothing added
                 lambda: gf.gf_rmsnorm_execute(plan, x.half(), w, out=x),                     # type
                 lambda: gf.gf_rmsnorm_execute(plan, x[:3], w, out=x),                        # size
                 lambda: gf.gf_rmsnorm_execute(plan, x.t().contiguous().t(), w, out=x),       # layout
                 lambda: gf.gf_rmsnorm_execute(plan, x.cpu(), w, out=x),
                 lambda: gf.gf_rmsnorm_execute(plan, x.data_ptr() + 2, w, out=x),             # alignment
                 lambda: gf.gf_rmsnorm_grad_execute(plan, x, x, w, None),
                 lambda: gf.gf_route_execute(plan, x, x, w),                                  # another plan's call
                 lambda: gf.gf_moe_combine_execute(plan, x, x, x, x),
                 lambda: gf.gf_plan_set_option(plan, gf.GF_OPT_KERNEL, 1)):
        with pytest.raises(gf.GfError):
            call()
    gf.gf_plan_set_option(plan, gf.GF_OPT_PDL, 0)
    assert gf.gf_plan_describe(plan)["launches"] == 1 and gf.gf_plan_status(plan) == gf.GF_OK
    plan.free()
