"""Column sums over very many rows (the gradients of a norm's weight and of a bias): no term is lost, and none counted twice."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_epilogue_tmem_gb300 as gf  # noqa: E402

MOST = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    yield
    torch.cuda.empty_cache()


def grad(r, d_out, w, d_x, rows, hidden, eps):
    plan = gf.gf_rmsnorm_plan(rows, hidden, gf.GF_BF16, eps)
    d_w = torch.empty(hidden, device="cuda")
    gf.gf_rmsnorm_grad_execute(plan, d_out, r, w, d_x, d_weight=d_w)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    plan.free()
    return d_w.double().cpu()


def near_sum(got, want):
    # At most 8192 terms of one sign in a row, 8 such sums of a CTA, a 32nd of at most 32768 CTAs' (4096 terms: of 131072),
    # 32 of those. A step is off by 2^-24 of its sum, of the last sum half that on average: (8192 + 8 + 1024 + 32) / 2 x
    # 2^-24 < 2^-11.8; a term by a few 2^-24 besides
    assert bool(((got - want).abs() <= want.abs() * 2.0 ** -11.4).all()), ((got - want) / want).tolist()


# rows of whole words (streamed) and others, shorter than a word and of several
@pytest.mark.parametrize("rows,hidden", [(2 ** 30 + 5, 8), (2 ** 30 + 3, 7), (2 ** 28 + 1, 24)])
def test_weight_gradient_of_equal_rows(rows, hidden):
    row = torch.linspace(0.7, 1.9, hidden).bfloat16()
    r = row.cuda().repeat(rows).view(rows, hidden)
    d = (row.flip(0) * 0.83).bfloat16()
    d_out = d.cuda().repeat(rows).view(rows, hidden)
    w = torch.ones(hidden, device="cuda").bfloat16()
    got = grad(r, d_out, w, d_out, rows, hidden, 0.25)
    h = row.double() / (row.double().square().mean() + 0.25).sqrt()
    near_sum(got, rows * d.double() * h)


@pytest.mark.parametrize("act", [gf.GF_ACT_NONE, gf.GF_ACT_RELU])
def test_bias_gradient_of_equal_rows(act):
    rows, cols = 2 ** 30 + 77, 8
    row = torch.linspace(0.7, 1.9, cols).bfloat16()
    d = row.cuda().repeat(rows).view(rows, cols)
    plan, bgrad = gf.gf_dact_bgrad_plan(rows, cols, gf.GF_BF16, act), torch.empty(cols, device="cuda")
    if act == gf.GF_ACT_NONE:
        gf.gf_dact_bgrad_execute(plan, d, bgrad=bgrad)
    else:
        gf.gf_dact_bgrad_execute(plan, d, d, d, bgrad)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    plan.free()
    near_sum(bgrad.double().cpu(), rows * row.double())


@pytest.mark.parametrize("rows,hidden", [(MOST, 1), (2 ** 30 + 5, 8)])
def test_weight_gradient_of_a_few_rows_among_the_most(rows, hidden):
    """All but a few gradients are 0: the sum is theirs alone, each once."""
    r = torch.ones(rows, hidden, dtype=torch.bfloat16, device="cuda")
    d_out = torch.zeros_like(r)
    at = [0, 1, 4095, 2 ** 20 + 1, 2 ** 29 - 1, 2 ** 29, 2 ** 30, rows - 2, rows - 1]
    for i, row in enumerate(at):
        d_out[row] = 2.0 ** i
    got = grad(r, d_out, torch.ones(hidden, device="cuda").bfloat16(), d_out, rows, hidden, 3.0)
    # 1 / sqrt(1 + 3): powers of two throughout, but for a step of the root
    assert bool(((got - (2.0 ** len(at) - 1) / 2).abs() <= 2.0 ** len(at) * 4 * 2.0 ** -24).all()), got.tolist()
