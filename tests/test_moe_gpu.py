"""Expert routing on the GPU: the sort, the copies of the tokens' rows and back,
and their gradients, against plain implementations in 64 bits (integers and
copies exactly)."""
import itertools

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_epilogue_tmem_gb300 as gf  # noqa: E402
from fp8_reference import quantize_reference  # noqa: E402

TDT = {gf.GF_F16: torch.float16, gf.GF_BF16: torch.bfloat16}
# unit roundoff of the outputs, and the largest rounding error below the
# smallest normal
ROUND = {gf.GF_F16: (2.0 ** -11, 2.0 ** -25), gf.GF_BF16: (2.0 ** -8, 0.0)}
DTYPES = [gf.GF_F16, gf.GF_BF16]

# tokens, topk, experts, hidden: one token and none; one expert; hidden that
# no vector divides, below one vector, below and above one block of 128; the
# single-launch sort and the two-launch one, chunks that end inside a warp,
# more experts than slots, the largest topk and number of experts
SHAPES = [
    (1, 1, 1, 1), (1, 8, 128, 5120), (0, 2, 4, 64), (3, 2, 4, 7), (17, 3, 5, 128), (64, 8, 128, 136),
    (33, 64, 70, 24), (500, 8, 60, 250), (513, 8, 1000, 16), (999, 6, 1024, 40), (5003, 2, 3, 33),
    (9001, 1, 1, 8), (4100, 5, 256, 72), (9000, 4, 130, 16), (4100, 8, 1024, 24), (33000, 1, 600, 8),
]


def routing(tokens, topk, experts, seed, drop):
    """Distinct experts a token where there are enough; dropped slots as -1 and as other ids outside."""
    rng = np.random.default_rng(seed)
    if topk <= experts:
        e = np.argsort(rng.random((tokens, experts)), axis=1)[:, :topk].astype(np.int32)
    else:
        e = rng.integers(0, experts, (tokens, topk), dtype=np.int32)
    bad = rng.random((tokens, topk)) < drop
    e[bad] = rng.choice(np.array([-1, experts, -2 ** 31, 2 ** 31 - 1], np.int64),
                        bad.sum()).astype(np.int32)
    return e


def sort_reference(e, experts):
    flat = e.reshape(-1).astype(np.int64)
    kept = np.flatnonzero((flat >= 0) & (flat < experts))
    order = kept[np.argsort(flat[kept], kind="stable")]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[kept], minlength=experts))])
    row_of = np.full(flat.size, -1, np.int64)
    row_of[order] = np.arange(order.size)
    slot_of = np.full(flat.size, -1, np.int64)
    slot_of[:order.size] = order
    return offsets, row_of.reshape(e.shape), slot_of


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def randn(*shape, seed, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def int_out(*shape):
    return torch.full(shape, 77, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("tokens,topk,experts,hidden", SHAPES)
@pytest.mark.parametrize("dtype,drop", [(gf.GF_F16, 0.0), (gf.GF_BF16, 0.2), (gf.GF_BF16, 1.0)])
def test_dispatch(tokens, topk, experts, hidden, dtype, drop):
    e = routing(tokens, topk, experts, 1, drop)
    offsets, row_of, slot_of = sort_reference(e, experts)
    kept, slots = offsets[-1], tokens * topk
    x = randn(tokens, hidden, seed=2, dtype=TDT[dtype])
    plan = gf.gf_moe_plan(tokens, topk, experts, hidden, dtype)
    o, r, s = int_out(experts + 1), int_out(tokens, topk), int_out(slots)
    rows = torch.full((slots, hidden), float("nan"), dtype=TDT[dtype], device="cuda")
    for copies in (True, False):  # with the rows, and the sort alone
        gf.gf_moe_dispatch_execute(plan, dev(e), x if copies else None, o, r, s,
                                   rows if copies else None)
        assert gf.gf_plan_status(plan) == gf.GF_OK
        assert np.array_equal(o.cpu().numpy(), offsets)
        assert np.array_equal(r.cpu().numpy(), row_of)
        assert np.array_equal(s.cpu().numpy(), slot_of)
        for t in (o, r, s):
            t.fill_(77)
    want = torch.zeros_like(rows)
    want[:kept] = x[dev(slot_of[:kept] // topk)]
    assert torch.equal(rows, want)
    fused = slots <= 49152 and slots * hidden <= 40 << 20
    assert gf.gf_plan_describe(plan)["launches"] == (1 if fused else 2)
    plan.free()


@pytest.mark.parametrize("tokens,topk,experts,hidden", [
    (1, 8, 128, 5120), (0, 2, 4, 64), (3, 2, 4, 16), (17, 3, 5, 128), (64, 8, 128, 144),
    (500, 8, 60, 1040), (999, 6, 1024, 528)])
@pytest.mark.parametrize("dtype,drop", [(gf.GF_F16, 0.0), (gf.GF_BF16, 0.3)])
def test_dispatch_fp8(tokens, topk, experts, hidden, dtype, drop):
    e = routing(tokens, topk, experts, 3, drop)
    offsets, row_of, slot_of = sort_reference(e, experts)
    kept, slots, blocks = offsets[-1], tokens * topk, -(-hidden // 128)
    x = randn(tokens, hidden, seed=4, dtype=TDT[dtype]) * 3
    if tokens > 3:
        x[1] = 0  # blocks of zeros
        x[2, 5] = float("inf")
        x[3, 6] = float("nan")
    plan = gf.gf_moe_plan(tokens, topk, experts, hidden, dtype)
    o, r, s = int_out(experts + 1), int_out(tokens, topk), int_out(slots)
    rows = torch.full((slots, hidden), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((slots, blocks), float("nan"), device="cuda")
    gf.gf_moe_dispatch_fp8_execute(plan, dev(e), x, o, r, s, rows, scale)
    assert np.array_equal(o.cpu().numpy(), offsets)
    assert np.array_equal(r.cpu().numpy(), row_of)
    assert np.array_equal(s.cpu().numpy(), slot_of)
    q, sc = quantize_reference(x.double().cpu().numpy(), 1)
    want = np.zeros((slots, hidden))
    want[:kept] = q[slot_of[:kept] // topk]
    want_scale = np.ones((slots, blocks))
    want_scale[:kept] = sc[slot_of[:kept] // topk]
    got = rows.view(torch.float8_e4m3fn).double().cpu().numpy()
    np.testing.assert_array_equal(got, want)
    assert np.array_equal(scale.cpu().numpy(), want_scale)
    plan.free()


def gathered(rows, row_of):
    """rows[row_of] in 64 bits, zeros where dropped: [tokens, topk, hidden]"""
    at = torch.from_numpy(row_of).cuda()
    got = rows.double()[at.clamp(min=0)]
    return torch.where((at >= 0)[:, :, None], got, 0.0)


@pytest.mark.parametrize("tokens,topk,experts,hidden",
                         [s for s in SHAPES if s[0] > 0] + [(2, 8, 16, 4096), (200, 4, 8, 2047)])
@pytest.mark.parametrize("dtype,drop", [(gf.GF_F16, 0.0), (gf.GF_BF16, 0.2), (gf.GF_F16, 1.0)])
def test_back_and_gradients(tokens, topk, experts, hidden, dtype, drop):
    """dispatch's gradient, combine and its two gradients. Each sum over topk
    slots has topk fp32 additions and as many products, the dot product over
    hidden as many; every output is rounded once."""
    e = routing(tokens, topk, experts, 5, drop)
    offsets, row_of, _ = sort_reference(e, experts)
    kept, slots = int(offsets[-1]), tokens * topk
    rows = randn(slots, hidden, seed=6, dtype=TDT[dtype])
    rows[kept:] = float("nan")  # rows without a slot are not read
    d_out = randn(tokens, hidden, seed=7, dtype=TDT[dtype])
    weight = torch.softmax(randn(tokens, topk, seed=8, dtype=torch.float32), 1)
    weight[torch.from_numpy(row_of).cuda() < 0] = float("nan")  # nor their weights
    u, tiny = ROUND[dtype]
    plan = gf.gf_moe_plan(tokens, topk, experts, hidden, dtype)
    o, r = dev(offsets.astype(np.int32)), dev(row_of.astype(np.int32))
    g = gathered(rows, row_of)
    w = torch.where(torch.from_numpy(row_of).cuda() >= 0, weight.double(), 0.0)

    def close(got, want, terms, magnitude, unit, least):
        # `terms` fp32 operations on values of total `magnitude`, one rounding
        bound = terms * 2.0 ** -24 * magnitude
        bound = bound + unit * (want.abs() + bound) + least
        off = (got.double() - want).abs()
        assert bool((off <= bound).all()), f"{(off - bound).max().item():.3e} over the bound"

    d_x = torch.full((tokens, hidden), float("nan"), dtype=TDT[dtype], device="cuda")
    gf.gf_moe_dispatch_grad_execute(plan, r, rows, d_x)
    close(d_x, g.sum(1), topk, g.abs().sum(1), u, tiny)

    out = torch.full((tokens, hidden), float("nan"), dtype=TDT[dtype], device="cuda")
    gf.gf_moe_combine_execute(plan, r, weight, rows, out)
    wg = w[:, :, None] * g
    close(out, wg.sum(1), 2 * topk, wg.abs().sum(1), u, tiny)

    d_rows = torch.full((slots, hidden), float("nan"), dtype=TDT[dtype], device="cuda")
    d_weight = torch.full((tokens, topk), float("nan"), device="cuda")
    gf.gf_moe_combine_grad_execute(plan, o, r, weight, rows, d_out, d_rows, d_weight)
    dots = g * d_out.double()[:, None, :]
    close(d_weight, dots.sum(2), 2 * hidden, dots.abs().sum(2), 0.0, 0.0)
    want = torch.zeros(slots + 1, hidden, dtype=torch.float64, device="cuda")
    at = torch.from_numpy(np.where(row_of < 0, slots, row_of)).cuda()
    want[at.reshape(-1)] = (w[:, :, None] * d_out.double()[:, None, :]).reshape(slots, hidden)
    want[slots] = 0
    close(d_rows, want[:slots], 1, want[:slots].abs(), u, tiny)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    plan.free()


def test_gradients_against_differences():
    """<grad, v> of loss = sum(c * combine(dispatch(x), weight)) along random
    directions v of x and of the weights, against the loss's own difference:
    the map is linear in each, so that the difference is exact up to rounding."""
    tokens, topk, experts, hidden = 300, 4, 16, 264
    e = dev(routing(tokens, topk, experts, 9, 0.1))
    plan = gf.gf_moe_plan(tokens, topk, experts, hidden, gf.GF_F16)
    c = randn(tokens, hidden, seed=10, dtype=torch.float16)
    weight = torch.rand(tokens, topk, device="cuda")
    o, r, s = int_out(experts + 1), int_out(tokens, topk), int_out(tokens * topk)
    rows = torch.empty(tokens * topk, hidden, dtype=torch.float16, device="cuda")
    out = torch.empty(tokens, hidden, dtype=torch.float16, device="cuda")

    def loss(x, w):
        gf.gf_moe_dispatch_execute(plan, e, x, o, r, s, rows)
        gf.gf_moe_combine_execute(plan, r, w, rows, out)
        return (c.double() * out.double()).sum().item()

    x = randn(tokens, hidden, seed=11, dtype=torch.float16)
    base = loss(x, weight)
    d_rows, d_w = torch.empty_like(rows), torch.empty_like(weight)
    gf.gf_moe_combine_grad_execute(plan, o, r, weight, rows, c, d_rows, d_w)
    d_x = torch.empty_like(x)
    gf.gf_moe_dispatch_grad_execute(plan, r, d_rows, d_x)
    # out, d_rows and d_x each carry a rounding of 2^-11 per element: errors of
    # random sign on sums of tokens * hidden terms of size about topk
    slack = 8 * 2.0 ** -11 * topk * (tokens * hidden) ** 0.5
    vx = torch.randint(-1, 2, x.shape, device="cuda").to(torch.float16) / 4
    x2 = (x + vx).to(torch.float16)
    step = x2.double() - x.double()
    assert abs(loss(x2, weight) - base - (d_x.double() * step).sum().item()) <= slack
    vw = torch.randint(-1, 2, weight.shape, device="cuda").float()
    w2 = weight + vw
    assert abs(loss(x, w2) - base - (d_w.double() * (w2.double() - weight.double())).sum().item()) <= slack
    plan.free()


def test_same_bits_every_time_and_on_other_streams():
    """Two plans on two streams, against the same calls one after the other."""
    tokens, topk, experts, hidden = 3000, 6, 40, 520
    e = dev(routing(tokens, topk, experts, 12, 0.05))
    x = randn(tokens, hidden, seed=13, dtype=torch.bfloat16)
    weight = torch.rand(tokens, topk, device="cuda")

    def step(plan, stream):
        bufs = [int_out(experts + 1), int_out(tokens, topk), int_out(tokens * topk),
                torch.empty(tokens * topk, hidden, dtype=torch.bfloat16, device="cuda"),
                torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda"),
                torch.empty(tokens * topk, hidden, dtype=torch.bfloat16, device="cuda"),
                torch.empty(tokens, topk, device="cuda")]
        o, r, s, rows, out, d_rows, d_w = bufs
        torch.cuda.synchronize()
        gf.gf_moe_dispatch_execute(plan, e, x, o, r, s, rows, stream=stream)
        gf.gf_moe_combine_execute(plan, r, weight, rows, out, stream=stream)
        gf.gf_moe_combine_grad_execute(plan, o, r, weight, rows, x, d_rows, d_w, stream=stream)
        return bufs

    plans = [gf.gf_moe_plan(tokens, topk, experts, hidden, gf.GF_BF16) for _ in range(2)]
    first = step(plans[0], torch.cuda.current_stream())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    both = [step(p, s) for p, s in zip(plans, streams)]
    torch.cuda.synchronize()
    for a, b in itertools.product([first], both):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_rows_past_32_bit_offsets():
    """tokens * topk * hidden passes 2^31 elements: the last rows are right."""
    tokens, topk, experts, hidden = 70000, 8, 16, 4096
    e = np.tile(np.arange(topk, dtype=np.int32), (tokens, 1))
    e[-1] = np.arange(8, 16)  # the last token alone has the last experts
    x = randn(tokens, hidden, seed=14, dtype=torch.bfloat16)
    plan = gf.gf_moe_plan(tokens, topk, experts, hidden, gf.GF_BF16)
    slots = tokens * topk
    assert slots * hidden > 2 ** 31
    o, r, s = int_out(experts + 1), int_out(tokens, topk), int_out(slots)
    rows = torch.empty(slots, hidden, dtype=torch.bfloat16, device="cuda")
    gf.gf_moe_dispatch_execute(plan, dev(e), x, o, r, s, rows)
    offsets, row_of, _ = sort_reference(e, experts)
    assert np.array_equal(r.cpu().numpy(), row_of)
    assert torch.equal(rows[-8:], x[-1:].expand(8, hidden))
    at = slots - 8 - 5
    assert torch.equal(rows[at], x[tokens - 2 - 4])  # expert 7's rows are tokens 0 .. tokens - 2
    d_x = torch.empty_like(x)
    gf.gf_moe_dispatch_grad_execute(plan, r, rows, d_x)
    assert torch.equal(d_x[-3:], (8 * x[-3:].float()).to(torch.bfloat16))
    weight = torch.full((tokens, topk), 0.5, device="cuda")
    d_rows, d_w = torch.empty_like(rows), torch.empty_like(weight)
    gf.gf_moe_combine_grad_execute(plan, o, r, weight, rows, x, d_rows, d_w)
    assert torch.equal(d_rows[-8:], (x[-1:].float() / 2).to(torch.bfloat16).expand(8, hidden))
    plan.free()


class Guarded:
    """n elements between two runs of canaries, 16-byte aligned."""

    def __init__(self, *shape, dtype):
        n = int(np.prod(shape))
        self.flat = torch.full((4096 + n + 4096,), 0x5A, dtype=torch.int32, device="cuda").view(torch.uint8)
        size = torch.empty(0, dtype=dtype).element_size()
        self.lo, self.hi = 4096, 4096 + n * size
        self.flat.fill_(0x5A)
        self.t = self.flat[self.lo:self.hi].view(dtype).view(*shape)

    def intact(self):
        return bool((self.flat[:self.lo] == 0x5A).all()) and bool((self.flat[self.hi:] == 0x5A).all())


@pytest.mark.parametrize("tokens,topk,experts,hidden", [
    (1, 3, 5, 1), (1, 1, 1, 7), (5, 2, 3, 15), (9, 5, 7, 33), (40, 8, 20, 2047), (700, 7, 9, 250), (33, 3, 40, 264), (1500, 3, 5, 13)])
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_no_stray_stores(tokens, topk, experts, hidden, drop):
    """Every output of every call between canaries, at widths that end inside a word."""
    slots = tokens * topk
    e = dev(routing(tokens, topk, experts, 21, drop))
    x = randn(tokens, hidden, seed=22, dtype=torch.float16)
    w = torch.rand(tokens, topk, device="cuda")
    f16, i32 = torch.float16, torch.int32
    o, r, s = Guarded(experts + 1, dtype=i32), Guarded(tokens, topk, dtype=i32), Guarded(slots, dtype=i32)
    rows, d_rows = Guarded(slots, hidden, dtype=f16), Guarded(slots, hidden, dtype=f16)
    out, d_x = Guarded(tokens, hidden, dtype=f16), Guarded(tokens, hidden, dtype=f16)
    d_w = Guarded(tokens, topk, dtype=torch.float32)
    plan = gf.gf_moe_plan(tokens, topk, experts, hidden, gf.GF_F16)
    gf.gf_moe_dispatch_execute(plan, e, x, o.t, r.t, s.t, rows.t)
    gf.gf_moe_combine_execute(plan, r.t, w, rows.t, out.t)
    gf.gf_moe_combine_grad_execute(plan, o.t, r.t, w, rows.t, x, d_rows.t, d_w.t)
    gf.gf_moe_dispatch_grad_execute(plan, r.t, d_rows.t, d_x.t)
    guarded = [o, r, s, rows, d_rows, out, d_x, d_w]
    if hidden % 16 == 0:
        q, sc = Guarded(slots, hidden, dtype=torch.uint8), Guarded(slots, -(-hidden // 128), dtype=torch.float32)
        gf.gf_moe_dispatch_fp8_execute(plan, e, x, o.t, r.t, s.t, q.t, sc.t)
        guarded += [q, sc]
    assert gf.gf_plan_status(plan) == gf.GF_OK
    assert all(g.intact() for g in guarded)
    plan.free()


def test_graph_capture():
    tokens, topk, experts, hidden = 700, 8, 32, 256
    plan = gf.gf_moe_plan(tokens, topk, experts, hidden, gf.GF_BF16)
    e = dev(routing(tokens, topk, experts, 15, 0.0))
    x = randn(tokens, hidden, seed=16, dtype=torch.bfloat16)
    o, r, s = int_out(experts + 1), int_out(tokens, topk), int_out(tokens * topk)
    rows = torch.empty(tokens * topk, hidden, dtype=torch.bfloat16, device="cuda")
    gf.gf_moe_dispatch_execute(plan, e, x, o, r, s, rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gf.gf_moe_dispatch_execute(plan, e, x, o, r, s, rows)
    e2 = routing(tokens, topk, experts, 17, 0.1)
    e.copy_(dev(e2))
    graph.replay()
    torch.cuda.synchronize()
    offsets, row_of, slot_of = sort_reference(e2, experts)
    assert np.array_equal(r.cpu().numpy(), row_of) and np.array_equal(s.cpu().numpy(), slot_of)
    plan.free()


def test_refusals():
    """Wrong tensors, missing pointers, misalignment and plans of another kind are refused before any launch."""
    t, k, e, h = 8, 2, 4, 24
    plan = gf.gf_moe_plan(t, k, e, h, gf.GF_BF16)
    expert, x = int_out(t, k), torch.zeros(t, h, dtype=torch.bfloat16, device="cuda")
    o, r, s = int_out(e + 1), int_out(t, k), int_out(t * k)
    rows = torch.zeros(t * k, h, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(t, k, device="cuda")
    good = [expert, x, o, r, s, rows]
    bad = [(0, expert.long()), (0, expert.cpu()), (0, None), (1, x.half()), (1, None), (5, None),
           (1, x.t()), (2, o[:-1]), (5, rows[:, :8]), (3, r.data_ptr() + 4)]
    for at, v in bad:
        args = list(good)
        args[at] = v
        with pytest.raises(gf.GfError) as err:
            gf.gf_moe_dispatch_execute(plan, *args)
        assert err.value.status == gf.GF_ERR_INVALID_VALUE
    # hidden % 16
    with pytest.raises(gf.GfError) as err:
        gf.gf_moe_dispatch_fp8_execute(plan, expert, x, o, r, s, rows.data_ptr(), w.data_ptr())
    assert err.value.status == gf.GF_ERR_UNSUPPORTED
    for call, args in ((gf.gf_moe_combine_execute, (r, None, rows, x)),
                       (gf.gf_moe_combine_execute, (r, w.half(), rows, x)),
                       (gf.gf_moe_dispatch_grad_execute, (r, rows, None)),
                       (gf.gf_moe_combine_grad_execute, (o, r, w, rows, x, rows, None)),
                       (gf.gf_moe_combine_grad_execute, (None, r, w, rows, x, rows, w))):
        with pytest.raises(gf.GfError) as err:
            call(plan, *args)
        assert err.value.status == gf.GF_ERR_INVALID_VALUE
    other = gf.gf_matmul_plan(64, 64, 64, gf.GF_BF16, gf.GF_EPILOG_NONE)
    with pytest.raises(gf.GfError):
        gf.gf_moe_combine_execute(other, r, w, rows, x)
    assert gf.lib().gf_moe_combine_execute(other.handle, *[r.data_ptr()] * 4, None) == \
        gf.GF_ERR_INVALID_VALUE
    with pytest.raises(gf.GfError):
        gf.gf_matmul_execute(plan, x, x, out=x)
    for option, value, status in ((gf.GF_OPT_SPLIT_K, 2, gf.GF_ERR_UNSUPPORTED),
                                  (gf.GF_OPT_PDL, 7, gf.GF_ERR_INVALID_VALUE),
                                  (99, 0, gf.GF_ERR_INVALID_VALUE)):
        with pytest.raises(gf.GfError) as err:
            gf.gf_plan_set_option(plan, option, value)
        assert err.value.status == status
    gf.gf_plan_set_option(plan, gf.GF_OPT_PDL, 0)
    torch.cuda.synchronize()
    assert bool((o == 77).all()) and bool((rows == 0).all())


@pytest.mark.parametrize("tokens,topk,experts,hidden", [
    (37, 11, 40, 2047), (29, 17, 64, 4999), (16, 2, 8, 9001), (61, 6, 60, 2050), (1, 64, 70, 1241), (3, 5, 9, 249),
    (130, 6, 16, 1025)])
@pytest.mark.parametrize("dtype,drop", [(gf.GF_F16, 0.0), (gf.GF_BF16, 0.3)])
def test_wide_odd_rows(tokens, topk, experts, hidden, dtype, drop):
    """Odd widths of several turns of a warp, and more slots than are in flight together."""
    test_back_and_gradients(tokens, topk, experts, hidden, dtype, drop)


@pytest.mark.parametrize("tokens,topk,experts,hidden", [(1201, 6, 60, 2047), (700, 8, 64, 4104), (4099, 2, 7, 1030)])
def test_dispatch_of_many_wide_rows(tokens, topk, experts, hidden):
    """The sort in a launch of its own before the copies of rows longer than one piece."""
    test_dispatch(tokens, topk, experts, hidden, gf.GF_BF16, 0.1)


@pytest.mark.parametrize("tokens,topk,experts,hidden", [
    (50001, 1, 600, 8), (12500, 4, 130, 16), (6300, 8, 1024, 24), (52000, 1, 3, 7), (2600, 8, 60, 2047), (700, 8, 64, 7504),
    (16400, 1, 5, 2563)])
def test_dispatch_in_two_launches(tokens, topk, experts, hidden):
    """More slots, or more to copy, than one launch does: counted by clusters, or by each CTA."""
    test_dispatch(tokens, topk, experts, hidden, gf.GF_BF16, 0.1)
    if hidden % 16 == 0:
        test_dispatch_fp8(tokens, topk, experts, hidden, gf.GF_F16, 0.1)


@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (700, 8, 64), (9000, 6, 1024), (12300, 8, 70), (33000, 4, 1024)])
def test_sort_alone(tokens, topk, experts):
    """The indexes without any copies, counted by each CTA and by clusters."""
    e = routing(tokens, topk, experts, 91, 0.1)
    offsets, row_of, slot_of = sort_reference(e, experts)
    kept = int(offsets[-1])
    plan = gf.gf_moe_plan(tokens, topk, experts, 64, gf.GF_F16)
    o, r, s = int_out(experts + 1), int_out(tokens, topk), int_out(tokens * topk)
    gf.gf_moe_dispatch_execute(plan, dev(e), None, o, r, s, None)
    assert np.array_equal(o.cpu().numpy(), offsets) and np.array_equal(r.cpu().numpy(), row_of)
    assert np.array_equal(s.cpu().numpy()[:kept], slot_of[:kept])
    plan.free()
