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
