"""What a plan of a block-scaled e4m3 product tells about itself (no kernel runs)."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_epilogue_tmem_gb300 as gf  # noqa: E402


def described(m, n, k, groups, kernel, epilog=gf.GF_FP8_EPILOG_NONE):
    plan = gf.gf_fp8_matmul_plan(m, n, k, groups, gf.GF_BF16, epilog)
    gf.gf_plan_set_option(plan, gf.GF_OPT_KERNEL, kernel)
    d = gf.gf_plan_describe(plan)
    plan.free()
    return d


@pytest.mark.parametrize("m,n,k,groups,kernel,splits", [
    # 32 tiles of 64 blocks on 152 CTAs: 128 of them, four a tile
    (1, 4096, 8192, 1, 1, 4), (16, 4096, 8192, 1, 1, 4), (64, 4096, 8192, 1, 2, 4),
    # 40 tiles of 136 blocks: 120 CTAs
    (1, 5120, 17408, 1, 1, 3),
    # six tiles of 50 blocks: 75 CTAs would have four blocks each, 72 are twelve a tile
    (40, 256, 6400, 1, 1, 12),
    # one and three blocks: shared by none
    (1, 128, 128, 1, 1, 1), (1, 128, 384, 1, 1, 1),
    # 94 tiles fill 61 % of a round; 32 tiles of 16 blocks would spare less than the join costs
    (1, 12000, 16384, 1, 1, 1), (1, 4096, 2048, 1, 1, 1),
    # 160 tiles of 64 blocks fill 53 % of two rounds of 152: 67 blocks a CTA, a tile falls to two at most
    (1, 20480, 8192, 1, 1, 2),
    (1, 4096, 0, 1, 1, 1), (0, 4096, 8192, 1, 1, 1),
    (16, 4096, 8192, 1, 3, 1), (16, 4096, 8192, 1, 4, 1),
    (16, 4096, 8192, 2, 1, 0), (64, 4096, 8192, 2, 2, 0), (64, 4096, 8192, 2, 3, 1)])
def test_k_splits(m, n, k, groups, kernel, splits):
    """The CTAs of a tile by the rule of the kernel for few rows, for 152 SMs."""
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("the numbers are for 152 SMs")
    assert described(m, n, k, groups, kernel)["k_splits"] == splits
