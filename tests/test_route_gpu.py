"""A router's choice on the GPU and its gradient against the definition in 64 bits: experts exactly."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_epilogue_tmem_gb300 as gf  # noqa: E402
from route_reference import route, route_grad  # noqa: E402

TDT = {gf.GF_F16: torch.float16, gf.GF_BF16: torch.bfloat16, gf.GF_F32: torch.float32}
ROUND = {gf.GF_F16: (2.0 ** -11, 2.0 ** -25), gf.GF_BF16: (2.0 ** -8, 0.0), gf.GF_F32: (2.0 ** -24, 2.0 ** -149)}
SOFTMAX, SIGMOID = gf.GF_SCORE_SOFTMAX, gf.GF_SCORE_SIGMOID
NAN, INF = float("nan"), float("inf")

# tokens, experts, topk, groups, topk_groups, group_best: one expert; fewer experts than lanes; groups of one and of
# sizes that no lanes divide; the most experts, groups and slots
SHAPES = [(1, 1, 1, 1, 1, 1), (5, 3, 3, 1, 1, 1), (0, 8, 2, 1, 1, 1), (67, 8, 2, 4, 2, 1), (130, 60, 6, 1, 1, 1), (130, 60, 6, 3, 2, 2),
          (99, 64, 8, 8, 8, 2), (41, 128, 8, 1, 1, 1), (300, 160, 6, 8, 3, 2), (257, 256, 8, 8, 4, 2), (77, 256, 8, 32, 4, 1),
          (33, 33, 4, 33 // 11, 2, 2), (19, 17, 5, 17, 9, 2), (31, 512, 33, 1, 1, 1), (7, 1000, 64, 4, 3, 2), (9, 1024, 10, 1, 1, 1),
          (5, 1023, 8, 3, 2, 2), (6, 1020, 8, 17, 5, 2), (12, 1024, 8, 32, 32, 2), (40, 2, 1, 2, 1, 2),
          # many tokens, eight lanes each: the last warp not full, every number of experts a lane, one group's lane that has all picks
          (2049, 8, 2, 1, 1, 1), (2500, 60, 6, 1, 1, 1), (2051, 64, 8, 8, 3, 2), (2048, 128, 16, 4, 2, 1), (3003, 160, 6, 8, 3, 2), (2100, 256, 8, 8, 1, 2),
          (2600, 256, 8, 8, 4, 2), (2050, 96, 3, 3, 2, 2)]


def logits_of(tokens, ld, seed, dtype, size=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (size * torch.randn(tokens, ld, generator=g, device="cuda")).to(TDT[dtype])


def call(logits, experts, topk, dtype, score, renorm, scale=1.0, bias=None, groups=1, topk_groups=1, best=1):
    tokens, ld = logits.shape
    plan = gf.gf_route_plan(tokens, experts, topk, dtype, score, renorm, scale, groups, topk_groups, best, ld)
    expert = torch.full((tokens, topk), 77, dtype=torch.int32, device="cuda")
    weight = torch.full((tokens, topk), NAN, device="cuda")
    gf.gf_route_execute(plan, logits, expert, weight, bias=bias)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    plan.free()
    return expert.cpu().numpy(), weight.double().cpu().numpy()


def check(logits, experts, topk, dtype, score, renorm, scale, bias, groups, topk_groups, best):
    expert, weight = call(logits, experts, topk, dtype, score, renorm, scale, bias, groups, topk_groups, best)
    b = None if bias is None else bias.double().cpu().numpy()
    l = logits[:, :experts].double().cpu().numpy()
    want, w = route(l, topk, score == SIGMOID, renorm, scale, b, groups, topk_groups, best)
    assert np.array_equal(expert, want), (np.argwhere(expert != want)[:4], expert[expert != want][:4], want[expert != want][:4])
    # exponentials, at most 1024 terms in 32 sums, a division
    assert np.all((np.isnan(weight) & np.isnan(w)) | (np.abs(weight - w) <= 2.0 ** -18 * np.abs(w)))


@pytest.mark.parametrize("tokens,experts,topk,groups,topk_groups,best", SHAPES)
@pytest.mark.parametrize("dtype,score,renorm,scale,biased,pad", [
    (gf.GF_F32, SIGMOID, True, 2.5, True, 0), (gf.GF_F32, SOFTMAX, False, 1.0, True, 3), (gf.GF_BF16, SOFTMAX, True, 1.0, False, 0),
    (gf.GF_F16, SIGMOID, False, -0.5, True, 8), (gf.GF_BF16, SIGMOID, True, 1.0, False, 1), (gf.GF_F16, SOFTMAX, False, 1.0, False, 5)])
def test_choice(tokens, experts, topk, groups, topk_groups, best, dtype, score, renorm, scale, biased, pad):
    logits = logits_of(tokens, experts + pad, 1, dtype)
    logits[:, experts:] = INF  # columns behind the experts are not looked at
    bias = None
    if biased:
        g = torch.Generator(device="cuda").manual_seed(2)
        bias = torch.randn(experts, generator=g, device="cuda") * (0.1 if score == SIGMOID else 0.3 / experts)
    check(logits, experts, topk, dtype, score, renorm, scale, bias, groups, topk_groups, best)


@pytest.mark.parametrize("dtype", [gf.GF_F32, gf.GF_BF16])
@pytest.mark.parametrize("score,biased", [(SOFTMAX, True), (SOFTMAX, False), (SIGMOID, True), (SIGMOID, False)])
@pytest.mark.parametrize("groups,topk_groups,best", [(1, 1, 1), (4, 2, 2), (4, 2, 1), (5, 2, 2)])
@pytest.mark.parametrize("tokens", [200, 2061])
def test_scores_next_to_each_other(dtype, score, biased, groups, topk_groups, best, tokens):
    """Equal logits, and logits a step of fp32 apart with biases that nearly undo them."""
    experts = 40
    rng = np.random.default_rng(3)
    l = rng.choice([0.0, -0.0, 0.5, 0.75, 1.0], (tokens, experts)).astype(np.float32)
    if dtype == gf.GF_F32:
        steps = rng.integers(-2, 3, l.shape) * (rng.random(l.shape) < 0.5)
        l = l * (1 + steps.astype(np.float32) * np.float32(2.0 ** -23))
    bias = None
    if biased:
        bias = rng.choice([0.0, 2.0 ** -24, -(2.0 ** -25), 0.125], experts).astype(np.float32)
        bias = torch.from_numpy(bias).cuda()
    logits = torch.from_numpy(l).cuda().to(TDT[dtype])
    check(logits, experts, 7, dtype, score, True, 1.0, bias, groups, topk_groups, best)


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("groups,topk_groups,best", [(1, 1, 1), (4, 2, 2), (4, 2, 1)])
@pytest.mark.parametrize("tokens", [12, 2060])
def test_masked_and_without_a_number(score, biased, groups, topk_groups, best, tokens):
    experts, topk = 64, 8
    logits = logits_of(tokens, experts, 4, gf.GF_F32)
    logits[0] = -INF                       # nothing left
    logits[1, 3:] = -INF                   # fewer than topk
    logits[2, ::2] = -INF
    logits[3] = torch.finfo(torch.float32).min
    logits[4, :60] = torch.finfo(torch.float32).min
    logits[5, 7] = NAN
    logits[6, 9] = INF
    logits[7, 5:9] = NAN
    logits[8, 16:] = -INF                  # whole groups
    logits[9, [0, 20, 40, 63]] = INF
    bias = None
    if biased:
        g = torch.Generator(device="cuda").manual_seed(5)
        bias = 0.1 * torch.randn(experts, generator=g, device="cuda")
        bias[11] = -INF                    # left out by the bias
        bias[12] = 1e6
    for renorm in (True, False):
        check(logits, experts, topk, gf.GF_F32, score, renorm, 1.0, bias, groups, topk_groups, best)


@pytest.mark.parametrize("tokens,experts,topk,pad", [(1, 1, 1, 0), (0, 8, 2, 0), (67, 8, 2, 4), (130, 60, 6, 0), (41, 128, 8, 8), (257, 256, 8, 0),
                                                      (31, 512, 33, 1), (7, 1000, 64, 0), (9, 1024, 10, 0),
                                                      (20001, 64, 8, 0), (130, 60, 9, 4), (1000, 120, 16, 8), (77, 512, 12, 0)])
@pytest.mark.parametrize("dtype,score,renorm,scale", [(gf.GF_F32, SIGMOID, True, 2.5), (gf.GF_F32, SOFTMAX, False, 1.0), (gf.GF_BF16, SOFTMAX, True, 1.0),
                                                      (gf.GF_F16, SIGMOID, False, -0.5)])
def test_gradient(tokens, experts, topk, pad, dtype, score, renorm, scale):
    logits = logits_of(tokens, experts + pad, 6, dtype)
    rng = np.random.default_rng(7)
    expert = np.argsort(rng.random((tokens, experts)), 1)[:, :topk].astype(np.int32)
    d_weight = rng.standard_normal((tokens, topk)).astype(np.float32)
    if tokens > 6:
        expert[1, 0], expert[2, :], expert[3, -1] = -1, -1, 2 ** 31 - 1
        d_weight[1, 0] = np.nan   # beside a slot without an expert
        expert[4, :] = expert[4, 0]  # the same expert in every slot
        logits[5, ::2] = -INF
        expert[5, 0] = 0          # a masked one
    plan = gf.gf_route_plan(tokens, experts, topk, dtype, score, renorm, scale, ld=experts + pad)
    d = torch.full_like(logits, NAN)
    gf.gf_route_grad_execute(plan, logits, torch.from_numpy(expert).cuda(), torch.from_numpy(d_weight).cuda(), d)
    plan.free()
    want, size = route_grad(logits[:, :experts].double().cpu().numpy(), expert, d_weight.astype(np.float64), score == SIGMOID, renorm, scale)
    got, (u, tiny) = d.double().cpu().numpy(), ROUND[dtype]
    assert np.all(np.abs(got[:, :experts] - want) <= u * np.abs(want) + 2.0 ** -18 * size + tiny)
    assert np.all(got[:, experts:] == 0)


@pytest.mark.parametrize("score,renorm", [(SOFTMAX, True), (SOFTMAX, False), (SIGMOID, True), (SIGMOID, False)])
def test_gradient_against_differences(score, renorm):
    logits = logits_of(1, 12, 8, gf.GF_F32)
    expert, _ = call(logits, 12, 4, gf.GF_F32, score, renorm, 1.5)
    g = np.random.default_rng(9).standard_normal((1, 4))
    plan = gf.gf_route_plan(1, 12, 4, gf.GF_F32, score, renorm, 1.5)
    d = torch.empty_like(logits)
    gf.gf_route_grad_execute(plan, logits, torch.from_numpy(expert).cuda(), torch.from_numpy(g.astype(np.float32)).cuda(), d)
    plan.free()
    l, step = logits.double().cpu().numpy(), 1e-4

    def loss(v):  # the choice held: smaller steps than the gaps between the scores
        e, w = route(v, 4, score == SIGMOID, renorm, 1.5)
        assert np.array_equal(e, expert)
        return (w * g).sum()

    for j in range(12):
        v = np.zeros_like(l)
        v[0, j] = step
        slope = (loss(l + v) - loss(l - v)) / (2 * step)
        assert abs(slope - float(d[0, j])) < 1e-6


def test_refusals():
    for args, status in (((4, 8, 2, gf.GF_F32, SIGMOID, True, 1.0, 3, 1, 1), gf.GF_ERR_INVALID_VALUE),     # groups of unequal size
                         ((4, 8, 5, gf.GF_F32, SIGMOID, True, 1.0, 2, 1, 1), gf.GF_ERR_INVALID_VALUE),     # topk in what stays
                         ((4, 64, 2, gf.GF_F32, SIGMOID, True, 1.0, 64, 4, 1), gf.GF_ERR_UNSUPPORTED),     # groups
                         ((4, 8, 2, gf.GF_F32, SIGMOID, True, NAN, 1, 1, 1), gf.GF_ERR_INVALID_VALUE),
                         ((4, 8, 2, gf.GF_F32, SIGMOID, True, 1.0, 1, 1, 1, 7), gf.GF_ERR_INVALID_VALUE)):  # ld
        with pytest.raises(gf.GfError) as e:
            gf.gf_route_plan(*args)
        assert e.value.status == status
    plan = gf.gf_route_plan(4, 8, 2, gf.GF_F32)
    l, e, w = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    for bad in (lambda: gf.gf_route_execute(plan, l.half(), e, w), lambda: gf.gf_route_execute(plan, l, e.long(), w),
                lambda: gf.gf_route_execute(plan, l, e, None), lambda: gf.gf_route_execute(plan, l, e, w, bias=l),
                lambda: gf.gf_route_execute(plan, l.data_ptr() + 4, e, w), lambda: gf.gf_route_grad_execute(plan, l, e, w, l.bfloat16()),
                lambda: gf.gf_moe_dispatch_execute(plan, e, None, e, e, e, None), lambda: gf.gf_plan_set_option(plan, gf.GF_OPT_SPLIT_K, 1)):
        with pytest.raises(gf.GfError):
            bad()
    plan.free()


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("pad", [0, 1])  # rows of whole 16-byte words or not
@pytest.mark.parametrize("topk", [1, 3])
def test_an_expert_alone_has_no_gradient(score, pad, topk):
    """Renormalised, the weight of a token's only expert is the scale whatever its logit is."""
    tokens, experts = 5000, 16
    logits = logits_of(tokens, experts + pad, 5, gf.GF_F32)
    g = torch.Generator(device="cuda").manual_seed(6)
    expert = torch.full((tokens, topk), -1, dtype=torch.int32, device="cuda")
    expert[:, topk // 2] = torch.randint(experts, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    d_weight, d_logits = torch.randn(tokens, topk, generator=g, device="cuda"), torch.empty_like(logits)
    plan = gf.gf_route_plan(tokens, experts, topk, gf.GF_F32, score, True, 2.5, 1, 1, 1, experts + pad)
    gf.gf_route_grad_execute(plan, logits, expert, d_weight, d_logits)
    assert torch.count_nonzero(d_logits) == 0
    plan.free()


# rows of words of 8, 4 and 2 bytes, with and without columns behind the experts
@pytest.mark.parametrize("tokens,experts,topk,pad", [(1001, 60, 6, 0), (999, 54, 8, 0), (500, 61, 9, 0), (333, 62, 16, 4), (77, 6, 3, 0), (18, 2, 1, 0),
                                                     (40, 505, 8, 3)])
@pytest.mark.parametrize("dtype,score", [(gf.GF_F32, SIGMOID), (gf.GF_BF16, SOFTMAX), (gf.GF_F16, SIGMOID)])
def test_gradient_of_ragged_rows(tokens, experts, topk, pad, dtype, score):
    test_gradient(tokens, experts, topk, pad, dtype, score, True, 1.5)
