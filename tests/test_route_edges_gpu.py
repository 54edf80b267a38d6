"""The router and its gradient where a token's scores vanish, or its logits lie far from 0: against the definition in 64 bits."""
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


def randn(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def choose(logits, experts, topk, dtype, score, renorm, scale, bias=None, groups=1, topk_groups=1, best=1):
    tokens, ld = logits.shape
    plan = gf.gf_route_plan(tokens, experts, topk, dtype, score, renorm, scale, groups, topk_groups, best, ld)
    expert = torch.full((tokens, topk), 77, dtype=torch.int32, device="cuda")
    weight = torch.full((tokens, topk), NAN, device="cuda")
    gf.gf_route_execute(plan, logits, expert, weight, bias=bias)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    plan.free()
    return expert, weight


def check_choice(logits, experts, topk, dtype, score, renorm, scale, bias=None, groups=1, topk_groups=1, best=1):
    expert, weight = choose(logits, experts, topk, dtype, score, renorm, scale, bias, groups, topk_groups, best)
    want, w = route(logits[:, :experts].double().cpu().numpy(), topk, score == SIGMOID, renorm, scale,
                    None if bias is None else bias.double().cpu().numpy(), groups, topk_groups, best)
    expert, weight = expert.cpu().numpy(), weight.double().cpu().numpy()
    assert np.array_equal(expert, want), (np.argwhere(expert != want)[:4], expert[expert != want][:4], want[expert != want][:4])
    # exponentials, at most 1024 terms in 32 sums, divisions
    assert np.all((np.isnan(weight) & np.isnan(w)) | (np.abs(weight - w) <= 2.0 ** -18 * np.abs(w)))
    return expert


def check_grad(logits, experts, expert, d_weight, dtype, score, renorm, scale):
    tokens, ld = logits.shape
    plan = gf.gf_route_plan(tokens, experts, expert.shape[1], dtype, score, renorm, scale, ld=ld)
    d = torch.full_like(logits, NAN)
    gf.gf_route_grad_execute(plan, logits, torch.from_numpy(expert.astype(np.int32)).cuda(), torch.from_numpy(d_weight).cuda(), d)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    plan.free()
    want, size = route_grad(logits[:, :experts].double().cpu().numpy(), expert, d_weight.astype(np.float64), score == SIGMOID, renorm, scale)
    got, (u, tiny) = d.double().cpu().numpy(), ROUND[dtype]
    assert np.all(np.abs(got[:, :experts] - want) <= u * np.abs(want) + 2.0 ** -18 * size + tiny)
    assert np.all(got[:, experts:] == 0)


# rows of 16-byte words, of words of 4 bytes and of single elements; more slots than the kernel of eight lanes has
@pytest.mark.parametrize("experts,topk,pad", [(32, 4, 0), (20, 20, 0), (30, 3, 0), (33, 5, 0), (64, 8, 3), (700, 8, 0)])
@pytest.mark.parametrize("dtype", [gf.GF_F32, gf.GF_BF16])
@pytest.mark.parametrize("score,renorm", [(SOFTMAX, True), (SOFTMAX, False), (SIGMOID, True), (SIGMOID, False)])
def test_gradient_of_tokens_without_experts(experts, topk, pad, dtype, score, renorm):
    """A token whose logits are all -inf has no gradient, with no slot filled and with masked experts in its slots."""
    tokens = 37
    logits = randn(tokens, experts + pad, seed=1).to(TDT[dtype])
    logits[::3] = -INF
    rng = np.random.default_rng(2)
    expert = np.argsort(rng.random((tokens, experts)), 1)[:, :topk].astype(np.int32)
    expert[0::6] = -1
    check_grad(logits, experts, expert, rng.standard_normal((tokens, topk)).astype(np.float32), dtype, score, renorm, 1.5)


@pytest.mark.parametrize("dtype,tokens", [(gf.GF_F32, 9), (gf.GF_BF16, 9), (gf.GF_F16, 2100)])
@pytest.mark.parametrize("score,renorm", [(SOFTMAX, True), (SOFTMAX, False), (SIGMOID, True), (SIGMOID, False)])
def test_slots_without_an_expert_beside_a_nan(dtype, tokens, score, renorm):
    """The weights of the experts chosen are NaN, those of the slots that find none 0."""
    experts, topk = 64, 8
    logits = torch.full((tokens, experts), -INF, device="cuda", dtype=TDT[dtype])
    logits[:, 11], logits[:, 30] = NAN, 0.5
    check_choice(logits, experts, topk, dtype, score, renorm, 1.0)


# every expert is wanted: as many as lanes, fewer, groups that do not fill their lanes, two slots a lane
@pytest.mark.parametrize("experts,groups,best", [(32, 1, 1), (20, 1, 1), (15, 5, 2), (12, 4, 1), (7, 7, 2), (33, 1, 1), (45, 3, 2), (60, 1, 1)])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_masked_tokens_that_want_every_expert(experts, groups, best, score, renorm):
    """Biases that are all equal leave nothing to compare but the masks: masked experts are left out, and those past the
    last expert are not looked at."""
    tokens = 70
    logits = randn(tokens, experts, seed=3)
    logits[::5] = -INF
    logits[1::5, ::2] = -INF
    logits[2::5] = NAN
    logits[3::5, experts // 2] = NAN
    logits[3::5, ::3] = -INF
    logits[4::10, experts - 1] = INF
    check_choice(logits, experts, experts, gf.GF_F32, score, renorm, 1.0, torch.zeros(experts, device="cuda"), groups, groups, best)


@pytest.mark.parametrize("experts,groups,kept", [(1024, 8, 4), (1024, 4, 2), (512, 8, 3), (256, 8, 4), (60, 5, 2)])
@pytest.mark.parametrize("offset", [-100.0, -50.0, 0.0, 50.0, 100.0, 1000.0])
def test_groups_of_logits_far_from_zero(experts, groups, kept, offset):
    """Softmax does not see what is added to all logits of a token; the groups' sums of two scores are compared as closely."""
    tokens, topk = 200000, 8
    logits = randn(tokens, experts, seed=int(offset) + 2000) + offset
    expert, _ = choose(logits, experts, topk, gf.GF_F32, SOFTMAX, True, 1.0, None, groups, kept, 2)
    for part in torch.arange(tokens, device="cuda").split(50000):
        l = logits[part].double()
        s = l.softmax(1).view(len(part), groups, -1)
        order = s.topk(2, 2).values.sum(2).sort(dim=1, descending=True, stable=True).indices[:, :kept]
        stays = torch.zeros(len(part), groups, dtype=torch.bool, device="cuda").scatter_(1, order, True)
        left = torch.where(stays.repeat_interleave(experts // groups, 1), l, -INF)
        want = left.sort(dim=1, descending=True, stable=True).indices[:, :topk]
        assert torch.equal(expert[part].long(), want), int((expert[part] != want).any(1).sum())


LOW = [-80.0, -86.0, -87.5, -90.0, -100.0, -103.5, -104.0, -120.0, -300.0, -600.0, -800.0, -1e5]


# a warp a token and eight lanes; an expert alone
@pytest.mark.parametrize("tokens,dtype", [(60, gf.GF_F32), (60, gf.GF_BF16), (2100, gf.GF_F16)])
@pytest.mark.parametrize("topk", [1, 8])
@pytest.mark.parametrize("renorm,scale", [(True, 2.5), (True, 1e6), (False, 2.5)])
def test_weights_of_low_sigmoid_scores(tokens, dtype, topk, renorm, scale):
    """Renormalised weights are ratios of scores, also where fp32 holds few of the scores' bits or none: e^l / (1 + e^l) of
    l down to -600, 0 in 64 bits from -745 on."""
    experts = 64
    base = torch.tensor(LOW, device="cuda").repeat(tokens // len(LOW) + 1)[:tokens, None]
    logits = (base + randn(tokens, experts, seed=7)).to(TDT[dtype])
    logits[:, 40] = base[:, 0].to(TDT[dtype]) - 40  # hardly any part in the sum
    logits[11, 9] = NAN
    if renorm:
        check_choice(logits, experts, topk, dtype, SIGMOID, renorm, scale)
    else:
        # as they are, scores are fp32's: of subnormal ones a step is 2^-149
        expert, weight = choose(logits, experts, topk, dtype, SIGMOID, renorm, scale)
        want, w = route(logits.double().cpu().numpy(), topk, True, renorm, scale)
        assert np.array_equal(expert.cpu().numpy(), want)
        weight = weight.double().cpu().numpy()
        assert np.all((np.isnan(weight) & np.isnan(w)) | (np.abs(weight - w) <= 2.0 ** -18 * w + 4 * scale * 2.0 ** -149))


@pytest.mark.parametrize("experts,topk,pad", [(64, 8, 0), (64, 1, 0), (61, 8, 0), (64, 20, 0), (64, 12, 2)])
@pytest.mark.parametrize("dtype", [gf.GF_F32, gf.GF_F16])
def test_gradient_of_low_sigmoid_scores(experts, topk, pad, dtype):
    tokens = 60
    base = torch.tensor(LOW, device="cuda").repeat(5)[:, None]
    logits = (base + randn(tokens, experts + pad, seed=8)).to(TDT[dtype])
    rng = np.random.default_rng(9)
    expert = np.argsort(rng.random((tokens, experts)), 1)[:, :topk]
    check_grad(logits, experts, expert, rng.standard_normal((tokens, topk)).astype(np.float32), dtype, SIGMOID, True, 2.5)


def test_a_token_does_not_depend_on_its_neighbours():
    """The same token among tokens of ordinary and of low scores, whose sums are formed otherwise: the same bits."""
    tokens, experts, topk = 4096, 64, 8
    logits = (randn(tokens, experts, seed=11) - 30).half()
    low = logits.clone()
    low[::2] -= 200
    for score in (SIGMOID, SOFTMAX):
        plan = gf.gf_route_plan(tokens, experts, topk, gf.GF_F16, score, True, 2.5)
        expert = torch.empty(tokens, topk, dtype=torch.int32, device="cuda")
        d_weight, got = randn(tokens, topk, seed=12), []
        for l in (logits, low):
            weight, d = torch.empty(tokens, topk, device="cuda"), torch.empty_like(l)
            gf.gf_route_execute(plan, l, expert, weight)
            gf.gf_route_grad_execute(plan, l, expert, d_weight, d)
            got.append((expert[1::2].clone(), weight[1::2], d[1::2]))
        plan.free()
        assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("tokens,dtype", [(60, gf.GF_F32), (2100, gf.GF_BF16)])
@pytest.mark.parametrize("base", [0.0, -8.0, -14.0, -20.0, -60.0, -80.0, -300.0])
def test_small_parts_of_low_sigmoid_sums(tokens, dtype, base):
    """Parts in the sum down to e^-70, of scores that fp32 holds in full, in part or not at all."""
    experts, topk = 64, 8
    logits = torch.full((tokens, experts), -INF, device="cuda")
    logits[:, 3::8] = base - torch.tensor([0.0, 5.0, 10.0, 20.0, 30.0, 40.0, 60.0, 70.0], device="cuda") - 0.5 * randn(tokens, 8, seed=13).abs()
    logits = logits.to(TDT[dtype])
    expert = check_choice(logits, experts, topk, dtype, SIGMOID, True, 2.5)
    rng = np.random.default_rng(14)
    check_grad(logits, experts, expert, rng.standard_normal((tokens, topk)).astype(np.float32), dtype, SIGMOID, True, 2.5)
