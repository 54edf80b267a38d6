"""The norm and the activation's gradient: calls of two threads, rows and values at the ends of their ranges."""
import sys
import threading

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_epilogue_tmem_gb300 as gf  # noqa: E402

TDT = {gf.GF_F16: torch.float16, gf.GF_BF16: torch.bfloat16}
NAN, INF = float("nan"), float("inf")


def randn(*shape, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def test_two_threads_with_their_own_plans():
    """Rows of other widths take the same kernel with other amounts of shared memory: one thread's call does not change
    what another's is launched with."""
    rows, calls = 1000, 20000
    failed, wrong = [], []
    start = threading.Barrier(4)

    def work(i, hidden, residual, grad):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                x, w = randn(rows, hidden, seed=i, dtype=torch.bfloat16), randn(hidden, seed=i + 9, dtype=torch.bfloat16)
                plan, out = gf.gf_rmsnorm_plan(rows, hidden, gf.GF_BF16), torch.empty_like(x)
                # addresses: as short a way to the call as there is
                xp, wp, op, on, res = x.data_ptr(), w.data_ptr(), out.data_ptr(), stream.cuda_stream, x.data_ptr() if residual else None

                def call():
                    if grad:
                        gf.gf_rmsnorm_grad_execute(plan, xp, xp, wp, op, d_residual=res, stream=on)
                    else:
                        gf.gf_rmsnorm_execute(plan, xp, wp, residual=res, out=op, stream=on)

                call()
                stream.synchronize()
                want = out.clone()
                start.wait(60)
                for _ in range(calls):
                    call()
                stream.synchronize()
                if not torch.equal(out, want):
                    wrong.append(i)
                plan.free()
        except Exception as e:  # a thread's error is the test's
            failed.append(f"{i}: {e}")
            start.abort()

    threads = [threading.Thread(target=work, args=(i, *a)) for i, a in
               enumerate([(2560, False, False), (8192, False, False), (2560, False, True), (8192, True, True)])]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert not failed and not wrong, (failed, wrong)


@pytest.mark.parametrize("dtype", [gf.GF_F16, gf.GF_BF16])
def test_relu_gradient_of_closed_units(dtype):
    """Where z > 0 does not hold, d_z and its part of the bias gradient are 0 whatever d_out is."""
    rows, cols = 300, 264
    d, z = randn(rows, cols, seed=1, dtype=TDT[dtype]), randn(rows, cols, seed=2, dtype=TDT[dtype])
    z[:, 0], z[:, 1] = 0.0, NAN
    closed = ~(z > 0)
    odd = torch.tensor([INF, -INF, NAN], device="cuda", dtype=TDT[dtype])[torch.arange(rows * cols, device="cuda").view(rows, cols) % 3]
    d = torch.where(closed, odd, d)
    plan = gf.gf_dact_bgrad_plan(rows, cols, dtype, gf.GF_ACT_RELU)
    d_z, bgrad = torch.empty_like(d), torch.empty(cols, device="cuda")
    gf.gf_dact_bgrad_execute(plan, d, z, d_z, bgrad)
    plan.free()
    want = torch.where(closed, 0.0, d.double())
    assert torch.equal(d_z.double(), want)
    # fp32 sums of at most 300 terms
    assert bool(((bgrad.double() - want.sum(0)).abs() <= want.abs().sum(0) * 300 * 2.0 ** -24).all())


@pytest.mark.parametrize("rows", [7, 6000])  # loaded by their CTA, and streamed
def test_e4m3_of_small_products(rows):
    """y of an ordinary size beside products r * weight near fp32's smallest: the factor of the row and the reciprocal of
    the scale are each within fp32, their product is not."""
    hidden = 256
    x = (randn(rows, hidden, seed=3) * 2.0 ** -55).bfloat16()
    w = ((1 + 0.3 * randn(hidden, seed=4)) * 2.0 ** -69).bfloat16()
    x[:, 5] = 0
    plan = gf.gf_rmsnorm_plan(rows, hidden, gf.GF_BF16, 0.0)
    q, scale = torch.empty(rows, hidden, dtype=torch.uint8, device="cuda"), torch.empty(rows, 2, device="cuda")
    gf.gf_rmsnorm_execute(plan, x, w, out8=q, out_scale=scale)
    plan.free()
    y = x.double() * w.double() / x.double().square().mean(1, keepdim=True).sqrt()
    top = y.abs().view(rows, 2, 128).amax(2)
    assert torch.equal(scale.double(), torch.exp2(torch.ceil(torch.log2(top / 448))))
    v, got = y / scale.double().repeat_interleave(128, 1), q.view(torch.float8_e4m3fn).double()
    # e4m3's rounding; and products of some 2^-124 are off by up to 2^-150, in steps of the scale (2^-76) and the
    # row's factor (2^55) 2^-19
    bound = torch.maximum(v.abs() * (2.0 ** -4 + 2.0 ** -17), torch.full_like(v, 2.0 ** -10 * (1 + 2.0 ** -17))) + 2.0 ** -18
    assert bool(((got - v).abs() <= bound).all())


def test_describe_is_what_runs():
    """The plans' grids, tiles and stages are those of the launches: tokens and rows of a CTA times CTAs that cover them,
    or a resident grid."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count

    def of(plan):
        d = gf.gf_plan_describe(plan)
        plan.free()
        return d

    # eight lanes a token: 16 tokens a CTA; a warp a token: 4, in a resident grid
    assert [of(gf.gf_route_plan(16384, 128, 8, gf.GF_BF16))[k] for k in ("tile_m", "grid")] == [16, 1024]
    d = of(gf.gf_route_plan(16384, 256, 8, gf.GF_F32, gf.GF_SCORE_SIGMOID, groups=8, topk_groups=4))
    assert d["tile_m"] == 4 and d["grid"] % sms == 0 and d["grid"] < 4096
    assert [of(gf.gf_route_plan(9, 256, 8, gf.GF_F32))[k] for k in ("tile_m", "grid")] == [4, 3]
    assert of(gf.gf_route_plan(0, 256, 8, gf.GF_F32))["grid"] == 0
    # few rows: one CTA each; many: a ring of several stages, all CTAs resident; rows that are not whole words: no ring
    assert [of(gf.gf_rmsnorm_plan(5, 5120, gf.GF_BF16))[k] for k in ("tile_m", "stages", "grid")] == [1, 0, 5]
    d = of(gf.gf_rmsnorm_plan(16384, 5120, gf.GF_BF16))
    assert d["tile_m"] == 1 and d["stages"] >= 2 and d["grid"] <= 5 * sms
    assert [of(gf.gf_rmsnorm_plan(5003, 2047, gf.GF_F16))[k] for k in ("tile_m", "stages", "grid")] == [1, 0, 5003]
    assert [of(gf.gf_rmsnorm_plan(7, 64, gf.GF_F16))[k] for k in ("tile_m", "grid")] == [4, 2]


def test_plans_of_the_forward_alone_hold_no_workspace():
    """A server keeps a plan for each number of tokens: without a gradient's call none holds memory for one."""
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    plans = [gf.gf_rmsnorm_plan(16384 + i, 5120, gf.GF_BF16) for i in range(64)]
    assert before - torch.cuda.mem_get_info()[0] < 16 << 20
    assert gf.gf_plan_describe(plans[0])["workspace_bytes"] <= 256
    for plan in plans:
        plan.free()


@pytest.mark.parametrize("rows,hidden", [(1000, 2048), (70, 999)])
def test_first_gradient_is_captured(rows, hidden):
    """The call that makes the workspace, in a graph: replayed, and the same bits as an ordinary one's."""
    x, d, w = randn(rows, hidden, seed=1).bfloat16(), randn(rows, hidden, seed=2).bfloat16(), randn(hidden, seed=3).bfloat16()
    plans = [gf.gf_rmsnorm_plan(rows, hidden, gf.GF_BF16) for _ in range(2)]
    outs = [(torch.zeros_like(x), torch.zeros(hidden, device="cuda")) for _ in plans]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gf.gf_rmsnorm_grad_execute(plans[0], d, x, w, outs[0][0], d_weight=outs[0][1])
    gf.gf_rmsnorm_grad_execute(plans[1], d, x, w, outs[1][0], d_weight=outs[1][1])
    for _ in range(2):
        outs[0][0].zero_(), outs[0][1].zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert gf.gf_plan_describe(plans[0])["workspace_bytes"] > 256
    # an eager call of the plan whose graph lives, without the weight's gradient, and with it
    gf.gf_rmsnorm_grad_execute(plans[0], d, x, w, outs[0][0])
    gf.gf_rmsnorm_grad_execute(plans[0], d, x, w, outs[0][0], d_weight=outs[0][1])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    del graph
    for plan in plans:
        plan.free()
