"""The norm, the router and the products with a residual as a program uses them together: the example's blocks and their
gradients against torch in 64 bits; captured and replayed, on other streams, without dependent launches; nothing
written outside their outputs."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import gemm_epilogue_tmem_gb300 as gf  # noqa: E402
from prenorm_block import DenseBlock, ExpertBlock  # noqa: E402
from route_reference import route, route_grad  # noqa: E402

U = 2.0 ** -8  # bfloat16


def randn(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def close(got, want, steps, why):
    """Norm of the difference within `steps` roundings to bfloat16 of the norm."""
    err = float((got.double() - want).norm() / want.norm())
    assert err <= steps * U, (why, err)


@pytest.mark.parametrize("tokens", [1, 37, 300])
def test_dense_block(tokens):
    block = DenseBlock(256, 512)
    x, stream, d_out = (randn(tokens, 256, seed=s) for s in (1, 2, 3))
    out = block.forward(x, stream)
    got = block.gradients(d_out)
    r = (x.float() + stream.float()).bfloat16().double().requires_grad_()
    w, b1, b2 = (t.double().requires_grad_() for t in (block.norm, block.b1, block.b2))
    y = r / (r.square().mean(1, keepdim=True) + 1e-6).sqrt() * w
    hid = torch.nn.functional.gelu(y @ block.w1.double().t() + b1, approximate="tanh")
    want = r + hid @ block.w2.double().t() + b2
    (want * d_out.double()).sum().backward()
    # roundings on the way: y, the argument of GELU or its value, out; back: d_z, d_y, d_x
    close(out, want.detach(), 4, "out")
    close(got["x"], r.grad, 6, "x")
    for name, t in (("norm", w), ("b1", b1), ("b2", b2)):
        close(got[name], t.grad, 6, name)


@pytest.mark.parametrize("tokens", [3, 200])
def test_expert_block(tokens):
    block = ExpertBlock(256, 128, experts=20, topk=3, groups=4, topk_groups=2)
    x, stream, d_out, d_experts = (randn(tokens, 256, seed=s) for s in (1, 2, 3, 4))
    out, r = block.forward(x, stream)
    p = block.plans[tokens]
    assert torch.equal(r, (x.float() + stream.float()).bfloat16())
    rd = r.double()
    y = rd / (rd.square().mean(1, keepdim=True) + 1e-6).sqrt() * block.norm.double()
    close(p["y"], y, 1, "y")
    close(p["logits"], p["y"].double() @ block.router.double().t(), 1, "logits")
    l = p["logits"][:, :20].double().cpu().numpy()
    expert, weight = route(l, 3, True, True, block.scale, block.balance.double().cpu().numpy(), 4, 2, 2)
    assert np.array_equal(p["expert"].cpu().numpy(), expert)
    assert np.allclose(p["weight"].cpu().numpy(), weight, rtol=2.0 ** -18, atol=0)

    def values(q, s):  # a scale for each 128 x 128 block
        return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)[:, :q.shape[1]].repeat_interleave(128, 2)[:, :, :q.shape[2]]

    gate, up, down = (values(*w) for w in (block.gate, block.up, block.down))
    want, e, w = torch.zeros(tokens, 256, dtype=torch.float64, device="cuda"), p["expert"].long(), p["weight"].double()
    for s in range(3):
        g = torch.einsum("th,tih->ti", p["y"].double(), gate[e[:, s]])
        u = torch.einsum("th,tih->ti", p["y"].double(), up[e[:, s]])
        want += w[:, s, None] * torch.einsum("ti,thi->th", torch.nn.functional.silu(g) * u, down[e[:, s]])
    close(out, want, 24, "out")  # y and h in e4m3: 2^-4 a value, of which some 1.5 remain after the sums
    got = block.gradients(d_out, d_experts)
    d_logits, size = route_grad(l, expert, got["weight"].double().cpu().numpy(), True, True, block.scale)
    assert np.all(np.abs(got["logits"][:, :20].double().cpu().numpy() - d_logits) <= U * np.abs(d_logits) + 2.0 ** -18 * size)
    assert bool((got["logits"][:, 20:] == 0).all())
    close(got["y"], got["logits"].double() @ block.router.double() + d_experts.double(), 1, "y")


def every_call(seed=0):
    """Calls of each operator on buffers of their own: (run, outputs) pairs."""
    calls = []
    bf = gf.GF_BF16

    def empty(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    for rows, hidden in ((5, 256), (700, 1024), (33, 250)):
        x, res, dy, w = (randn(*s, seed=seed + i) for i, s in enumerate([(rows, hidden)] * 3 + [(hidden,)]))
        plan = gf.gf_rmsnorm_plan(rows, hidden, bf)
        r, out, d_x, d_w = empty(rows, hidden), empty(rows, hidden), empty(rows, hidden), empty(hidden, dtype=torch.float32)
        calls.append((plan, lambda plan=plan, x=x, w=w, res=res, r=r, out=out, **k: gf.gf_rmsnorm_execute(plan, x, w, residual=res, residual_out=r, out=out, **k), [r, out]))
        calls.append((plan, lambda plan=plan, x=x, w=w, res=res, dy=dy, d_x=d_x, d_w=d_w, **k: gf.gf_rmsnorm_grad_execute(plan, dy, x, w, d_x, d_weight=d_w, d_residual=res, **k), [d_x, d_w]))
        if hidden % 16 == 0:
            q, s = empty(rows, hidden, dtype=torch.uint8), empty(rows, -(-hidden // 128), dtype=torch.float32)
            calls.append((plan, lambda plan=plan, x=x, w=w, q=q, s=s, **k: gf.gf_rmsnorm_execute(plan, x, w, out8=q, out_scale=s, **k), [q, s]))
    for tokens, experts, groups, biased in ((3, 60, 1, True), (2500, 64, 1, False), (2100, 128, 8, True)):
        l = randn(tokens, experts, seed=seed + 20)
        bias = 0.1 * torch.randn(experts, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") if biased else None
        plan = gf.gf_route_plan(tokens, experts, 4, bf, gf.GF_SCORE_SIGMOID, groups=groups, topk_groups=max(1, groups // 2))
        e, w, dw, dl = empty(tokens, 4, dtype=torch.int32), empty(tokens, 4, dtype=torch.float32), randn(tokens, 4, seed=9).float(), empty(tokens, experts)
        calls.append((plan, lambda plan=plan, l=l, e=e, w=w, bias=bias, **k: gf.gf_route_execute(plan, l, e, w, bias=bias, **k), [e, w]))
        calls.append((plan, lambda plan=plan, l=l, e=e, dw=dw, dl=dl, **k: gf.gf_route_grad_execute(plan, l, e, dw, dl, **k), [dl]))
    for m, n, k_, act in ((1, 1024, 2048, gf.GF_ACT_NONE), (48, 264, 4096, gf.GF_ACT_SILU), (300, 520, 512, gf.GF_ACT_GELU), (4096, 2560, 2048, gf.GF_ACT_RELU)):
        a, b, res, bias = randn(m, k_, seed=seed + 30), randn(n, k_, seed=seed + 31) / 32, randn(m, n, seed=seed + 32), randn(n, seed=seed + 33)
        plan = gf.gf_matmul_residual_plan(m, n, k_, bf, act, gf.GF_B_NK)
        out, z = empty(m, n), empty(m, n)
        calls.append((plan, lambda plan=plan, a=a, b=b, res=res, out=out, bias=bias, z=z, **k: gf.gf_matmul_residual_execute(plan, a, b, res, out, bias=bias, z_out=z, **k), [out, z]))
    dy, z = randn(515, 264, seed=seed + 40), randn(515, 264, seed=seed + 41)
    plan, d_z, bg = gf.gf_dact_bgrad_plan(515, 264, bf, gf.GF_ACT_GELU), empty(515, 264), empty(264, dtype=torch.float32)
    calls.append((plan, lambda plan=plan, **k: gf.gf_dact_bgrad_execute(plan, dy, z=z, d_z=d_z, bgrad=bg, **k), [d_z, bg]))
    return calls


def run_all(calls, **k):
    for plan, run, _ in calls:
        run(**k)
    torch.cuda.synchronize()
    for plan, _, _ in calls:
        assert gf.gf_plan_status(plan) == gf.GF_OK
    return [o.clone() for _, _, outs in calls for o in outs]


def same(a, b):
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def clear(calls):
    for _, _, outs in calls:
        for o in outs:
            o.fill_(0)
    torch.cuda.synchronize()


def test_captured_replayed_streams_and_plain_launches():
    calls = every_call()
    want = run_all(calls)
    clear(calls)
    side = torch.cuda.Stream()
    same(run_all(calls, stream=side), want)
    clear(calls)
    with torch.cuda.stream(side):
        for _, run, _ in calls:
            run()
    same(run_all([]) or [o.clone() for _, _, outs in calls for o in outs], want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _, run, _ in calls:
            run()
        for _, run, _ in calls:
            run()
    for _ in range(2):
        clear(calls)
        graph.replay()
        torch.cuda.synchronize()
        same([o for _, _, outs in calls for o in outs], want)
    for plan, _, _ in calls:
        gf.gf_plan_set_option(plan, gf.GF_OPT_PDL, 0)
    clear(calls)
    same(run_all(calls), want)


def test_two_streams_at_once():
    """The same operators with plans of their own on two streams."""
    a, b = every_call(), every_call(seed=100)
    want_a, want_b = run_all(a), run_all(b)
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        clear(a + b)
        for (_, ra, _), (_, rb, _) in zip(a, b):
            ra(stream=s[0])
            rb(stream=s[1])
        torch.cuda.synchronize()
        same([o for _, _, outs in a for o in outs], want_a)
        same([o for _, _, outs in b for o in outs], want_b)


@pytest.mark.parametrize("rows,hidden", [(1, 5), (7, 33), (350, 1000), (311, 4096), (2, 20002)])
def test_nothing_outside_the_outputs(rows, hidden):
    """Outputs between zones of a pattern, 16 bytes on: neither zone changes."""
    count, zone = rows * hidden, 64

    def guarded(n, dtype):
        whole = torch.full((n + 2 * zone,), 1.5, device="cuda").to(dtype)
        return whole, whole[zone:zone + n]

    x, res, dy, w = (randn(*s, seed=i) for i, s in enumerate([(rows, hidden)] * 3 + [(hidden,)]))
    plan = gf.gf_rmsnorm_plan(rows, hidden, gf.GF_BF16)
    zones = [guarded(count, torch.bfloat16) for _ in range(3)] + [guarded(hidden, torch.float32)]
    (_, r), (_, out), (_, d_x), (_, d_w) = zones
    gf.gf_rmsnorm_execute(plan, x, w, residual=res, residual_out=r, out=out)
    gf.gf_rmsnorm_grad_execute(plan, dy, x, w, d_x, d_weight=d_w, d_residual=res)
    if hidden % 8 == 0:
        z_plan = gf.gf_dact_bgrad_plan(rows, hidden, gf.GF_BF16, gf.GF_ACT_SILU)
        zones += [guarded(count, torch.bfloat16), guarded(hidden, torch.float32)]
        gf.gf_dact_bgrad_execute(z_plan, dy, z=x, d_z=zones[-2][1], bgrad=zones[-1][1])
        m_plan = gf.gf_matmul_residual_plan(rows, hidden, 64, gf.GF_BF16, gf.GF_ACT_SILU)
        zones += [guarded(count, torch.bfloat16), guarded(count, torch.bfloat16)]
        gf.gf_matmul_residual_execute(m_plan, randn(rows, 64, seed=7), randn(64, hidden, seed=8), res, zones[-2][1], z_out=zones[-1][1])
    for kept in range(1, 3):
        e_plan = gf.gf_route_plan(rows, min(hidden, 1000), kept, gf.GF_BF16, ld=hidden)
        zones += [guarded(rows * kept, torch.int32), guarded(rows * kept, torch.float32), guarded(count, torch.bfloat16)]
        gf.gf_route_execute(e_plan, x, zones[-3][1], zones[-2][1])
        gf.gf_route_grad_execute(e_plan, x, zones[-3][1], zones[-2][1], zones[-1][1])
    torch.cuda.synchronize()
    for whole, inner in zones:
        edge = torch.cat([whole[:zone], whole[zone + inner.numel():]])
        assert bool((edge == torch.full_like(edge, 1.5)).all())
