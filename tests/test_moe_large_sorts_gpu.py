"""Expert routing at the sizes where the sort's launch or its indexes change."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_epilogue_tmem_gb300 as gf  # noqa: E402
import test_moe_gpu as moe  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def check_dispatch(tokens, topk, experts, hidden, copies):
    """The indexes, and the rows where `copies`, against torch's stable sort; some slots are dropped."""
    expert = torch.randint(-1, experts, (tokens, topk), dtype=torch.int32, device="cuda")
    flat = expert.flatten().long()
    kept = int((flat >= 0).sum())
    order = torch.argsort(torch.where(flat < 0, experts, flat), stable=True)[:kept]
    i32 = dict(dtype=torch.int32, device="cuda")
    offsets, row_of, slot_of = torch.empty(experts + 1, **i32), torch.empty(tokens, topk, **i32), torch.empty(tokens * topk, **i32)
    x = torch.randn(tokens, hidden, device="cuda").half() if copies else None
    rows = torch.empty(tokens * topk, hidden, dtype=torch.half, device="cuda") if copies else None
    plan = gf.gf_moe_plan(tokens, topk, experts, hidden, gf.GF_F16)
    gf.gf_moe_dispatch_execute(plan, expert, x, offsets, row_of, slot_of, rows)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    assert torch.equal(slot_of[:kept].long(), order) and bool((slot_of[kept:] == -1).all())
    want = torch.full_like(flat, -1)
    want[order] = torch.arange(kept, device="cuda")
    assert torch.equal(row_of.flatten().long(), want)
    assert int(offsets[0]) == 0
    assert torch.equal(offsets[1:].long(), torch.cumsum(torch.bincount(flat[flat >= 0], minlength=experts), 0))
    if copies:
        assert torch.equal(rows[:kept], x[order // topk]) and not bool(rows[kept:].any())
    described = gf.gf_plan_describe(plan)
    plan.free()
    return described


@pytest.mark.parametrize("tokens,topk,experts,hidden,copies", [
    (19000, 8, 1024, 8, 0), (18900, 8, 1024, 16, 1), (48032, 4, 1002, 8, 0), (361700, 1, 900, 8, 1), (24320, 8, 1000, 8, 0)])
def test_first_call_of_a_process(tokens, topk, experts, hidden, copies):
    """Tables of a few bytes less than 48 KB, with the rows of a chunk's slots among them: with what the kernel holds
    besides they need the larger limit, which no earlier call has asked for."""
    call = f"import test_moe_large_sorts_gpu as t; t.check_dispatch({tokens}, {topk}, {experts}, {hidden}, {copies}); print('right')"
    path = os.pathsep.join([ROOT, os.path.join(ROOT, "tests"), os.environ.get("PYTHONPATH", "")])
    r = subprocess.run([sys.executable, "-c", call], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": path})
    assert r.returncode == 0 and r.stdout.strip() == "right", r.stderr[-2000:]


@pytest.mark.parametrize("tokens,topk,experts,hidden,copies", [
    (700001, 1, 1024, 8, 1), (1300001, 1, 3, 8, 0), (1300001, 1, 1024, 8, 1), (80000, 17, 60, 8, 1), (22000, 64, 70, 16, 0),
    (1 << 20, 8, 256, 8, 0)])
def test_chunks_do_not_grow_in_number(tokens, topk, experts, hidden, copies):
    """However many slots: every CTA or cluster counts them all, so that their number must not grow with the slots."""
    described = check_dispatch(tokens, topk, experts, hidden, copies)
    assert described["grid"] <= 2 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("experts,period", [(3, 3), (3, 4), (5, 64)])
def test_most_slots(experts, period):
    """2^31 - 1 slots, none dropped, a quarter and nearly all: indexes that pass 32 bits with the threads' stride. Slot i
    has expert i % period. The array before slot_of, as far as a negative 32-bit index reaches, stays as it is."""
    slots = 2 ** 31 - 1
    expert = torch.arange(slots, dtype=torch.int32, device="cuda").remainder_(period)
    offsets = torch.full((experts + 1,), 77, dtype=torch.int32, device="cuda")
    row_of = torch.full((slots,), 77, dtype=torch.int32, device="cuda")
    flat = torch.full((2 ** 31 + slots,), 77, dtype=torch.int32, device="cuda")
    slot_of = flat[2 ** 31:]
    plan = gf.gf_moe_plan(slots, 1, experts, 8, gf.GF_F16)
    gf.gf_moe_dispatch_execute(plan, expert, None, offsets, row_of, slot_of, None)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    plan.free()
    del expert
    counts = [(slots - e + period - 1) // period for e in range(experts)]
    starts = [sum(counts[:e]) for e in range(experts + 1)]
    assert offsets.tolist() == starts
    for e in range(period):
        if e < experts:
            rows = torch.arange(starts[e], starts[e + 1], dtype=torch.int32, device="cuda")
            assert torch.equal(row_of[e::period], rows)
            assert torch.equal(slot_of[starts[e]:starts[e + 1]], rows.sub_(starts[e]).mul_(period).add_(e))
        else:
            assert bool((row_of[e::period] == -1).all())
    assert bool((slot_of[starts[-1]:] == -1).all())
    assert bool((flat[:2 ** 31] == 77).all())


@pytest.mark.parametrize("tokens", [1, 2, 7, 20, 76])
@pytest.mark.parametrize("hidden", [9216, 16400, 16383, 32784, 33001, 65536])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_long_rows_of_few_tokens(tokens, hidden, drop):
    """Several CTAs share the copies of a token's row, and what is cleared behind the last."""
    moe.test_dispatch(tokens, 3, 9, hidden, gf.GF_BF16, drop)
    if hidden % 16 == 0:
        moe.test_dispatch_fp8(tokens, 3, 9, hidden, gf.GF_F16, drop)


@pytest.mark.parametrize("experts", [3, 128, 512, 1024])
@pytest.mark.parametrize("copies", [0, 1])
@pytest.mark.parametrize("more", [0, 1])
def test_either_way_of_counting(experts, copies, more):
    """On both sides of the number of slots from which on clusters of CTAs share the counting."""
    slots = (24576 + 32 * experts if copies else 49152 + 64 * experts) + more
    check_dispatch(slots, 1, experts, 2048 if copies else 8, copies)
