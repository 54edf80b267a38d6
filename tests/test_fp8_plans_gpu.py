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


# The kernel is the one whose expected time is the least: start + block * (k-blocks one after the other on an SM) +
# round * (tiles one after the other), us; 16-row tiles, 64-row tiles, single CTA, CTA pair; plain, and SwiGLU.
PACE = [[(4.0, 0.22, 0.8), (4.0, 0.29, 1.2), (3.4, 0.38, 2.8), (4.2, 0.34, 2.8)],
        [(4.0, 0.32, 3.0), (4.0, 0.75, 7.0), (4.6, 0.35, 3.0), (4.8, 0.33, 3.6)]]
ROWS = (16, 64, 128, 256)


def expected_times(m, n, k, groups, dual, sms, pairs):
    times = []
    for kernel, rows in enumerate(ROWS):
        cols = 128 if kernel < 2 or dual else 256
        row_tiles = -(-m // rows) if groups == 1 else groups * max(1.0, m / groups / rows + 0.4)
        each = row_tiles * -(-n // cols) / (pairs if kernel == 3 else sms)
        whole = -(-each // 1)
        rounds = whole if groups == 1 else max(1.0, each)
        blocks = rounds * -(-k // 128)
        if kernel < 2 and 100 * each < (65 if whole > 1 else 60) * whole:
            blocks = min(blocks, each * -(-k // 128) + (12 if dual else 15 if kernel == 0 else 20))
        start, block, per_round = PACE[dual][kernel]
        times.append(start + block * blocks + per_round * rounds)
    return times


@pytest.mark.parametrize("groups", [1, 8, 64])
@pytest.mark.parametrize("m", [1, 16, 48, 100, 256, 700, 2048, 8192, 40000])
def test_the_kernel_is_the_one_of_the_least_expected_time(m, groups):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    pairs = described(4096, 4096, 512, 1, 4)["grid"] // 2
    for n in (128, 1424, 4096, 17408):
        for k in (512, 2048, 8192):
            for dual in (0, 1):
                times = expected_times(m, n, k, groups, dual, sms, pairs)
                least, second = sorted(times)[:2]
                if second - least < 1e-9:  # a tie that rounding may break
                    continue
                d = described(m, n, k, groups, 0, dual)
                assert d["tile_m"] == ROWS[times.index(least)], (n, k, dual, times)


@pytest.mark.parametrize("m,n,k,groups,rows", [
    (8, 17408, 8192, 1, 16), (48, 9000, 8192, 1, 64), (256, 4096, 8192, 1, 64), (256, 17408, 8192, 1, 256),
    (64 * 64, 4096, 2048, 64, 128), (64 * 256, 4096, 2048, 64, 128), (8 * 1024, 4096, 16384, 8, 256)])
def test_the_kernel_measured_fastest(m, n, k, groups, rows):
    """Products whose times on all four kernels stand beside the rule."""
    assert described(m, n, k, groups, 0)["tile_m"] == rows
