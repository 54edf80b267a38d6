"""e4m3 quantisation (exactly) and the block-scaled e4m3 products (within the
error bound of their sums) on the GPU, against 64-bit references."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import gemm_epilogue_tmem_gb300 as gf  # noqa: E402
from fp8_reference import quantize_reference  # noqa: E402

TDT = {gf.GF_F16: torch.float16, gf.GF_BF16: torch.bfloat16}
ROUND = {gf.GF_F16: (2.0 ** -11, 2.0 ** -25), gf.GF_BF16: (2.0 ** -8, 0.0)}
KERNELS = [0, 1, 2, 3, 4]  # GF_OPT_KERNEL


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------- quantisation
@pytest.mark.parametrize("m,k", [(1, 16), (1, 5120), (3, 144), (16, 2048), (127, 128), (128, 400),
                                 (300, 1040), (1000, 272), (4096, 64)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [gf.GF_F16, gf.GF_BF16])
def test_quantize(m, k, block_rows, dtype):
    x = (torch.randn(m, k, generator=gen(1), device="cuda") *
         torch.exp2(torch.randint(-12, 8, (m, 1), generator=gen(2), device="cuda").float()))
    x = x.to(TDT[dtype])
    q = torch.full((m, k), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((-(-m // block_rows), -(-k // 128)), float("nan"), device="cuda")
    gf.gf_fp8_quantize(m, k, dtype, block_rows, x, q, s)
    want, scale = quantize_reference(x.double().cpu().numpy(), block_rows)
    assert np.array_equal(s.double().cpu().numpy(), scale)
    np.testing.assert_array_equal(q.view(torch.float8_e4m3fn).double().cpu().numpy(), want)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [gf.GF_F16, gf.GF_BF16])
def test_quantize_edges(block_rows, dtype):
    """Zeros, the type's largest and smallest values, infinities and NaN, maxima
    on both sides of 448 2^e, ties."""
    info = torch.finfo(TDT[dtype])
    rows = [torch.zeros(128), torch.full((128,), info.max), torch.full((128,), info.tiny),
            torch.full((128,), info.smallest_normal / 16 if dtype == gf.GF_F16 else 1e-40)]
    special = torch.randn(128, generator=torch.Generator().manual_seed(3))
    special[5], special[9], special[77] = float("inf"), -float("inf"), float("nan")
    rows += [special, torch.full((128,), float("nan")), torch.full((128,), -float("inf"))]
    for top in (448.0, 450.0, 446.0, 0.4375, 0.43774, 1.75, 1.7578125):
        ties = (torch.arange(128).float() * 2 + 1) / 16 * (top / 448)
        ties[0] = -top
        rows.append(ties)
    x = torch.stack(rows)
    if block_rows == 128:
        x = x.repeat_interleave(128, 0)
    x = x.to(TDT[dtype]).cuda().contiguous()
    m, k = x.shape
    q = torch.empty((m, k), dtype=torch.uint8, device="cuda")
    s = torch.empty((m // block_rows, 1), device="cuda")
    gf.gf_fp8_quantize(m, k, dtype, block_rows, x, q, s)
    want, scale = quantize_reference(x.double().cpu().numpy(), block_rows)
    assert np.array_equal(s.double().cpu().numpy(), scale)
    np.testing.assert_array_equal(q.view(torch.float8_e4m3fn).double().cpu().numpy(), want)


def test_scales_at_any_fp32_address():
    """Scales that begin at any 4-byte address: quantised into, and read from, parts of larger arrays."""
    m, n, k = 40, 136, 272
    x = torch.randn(m, k, generator=gen(4), device="cuda").half()
    w = torch.randn(n, k, generator=gen(5), device="cuda").half()
    qa, qb = torch.empty(m, k, dtype=torch.uint8, device="cuda"), torch.empty(n, k, dtype=torch.uint8, device="cuda")
    plan = gf.gf_fp8_matmul_plan(m, n, k, 1, gf.GF_F16)
    outs = []
    for lead in (0, 1, 3):
        sa, sb = torch.full((lead + m * 3 + 5,), 7.0, device="cuda"), torch.full((lead + 6 + 5,), 7.0, device="cuda")
        a, b = sa[lead:lead + m * 3], sb[lead:lead + 6]
        gf.gf_fp8_quantize(m, k, gf.GF_F16, 1, x, qa, a)
        gf.gf_fp8_quantize(n, k, gf.GF_F16, 128, w, qb, b)
        assert bool((sa[:lead] == 7).all() and (sa[lead + m * 3:] == 7).all() and (sb[lead + 6:] == 7).all())
        outs.append(torch.empty(m, n, dtype=torch.half, device="cuda"))
        gf.gf_fp8_matmul_execute(plan, qa, a, qb, b, out=outs[-1])
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    plan.free()


def test_quantize_refusals():
    x = torch.zeros(4, 32, dtype=torch.half, device="cuda")
    q, s = torch.zeros(4, 32, dtype=torch.uint8, device="cuda"), torch.zeros(4, 1, device="cuda")
    for args, status in (((4, 24, gf.GF_F16, 1, x.data_ptr(), q.data_ptr(), s), gf.GF_ERR_UNSUPPORTED),
                         ((4, 32, gf.GF_F16, 2, x, q, s.data_ptr()), gf.GF_ERR_INVALID_VALUE),
                         ((4, 32, 5, 1, x, q, s), gf.GF_ERR_INVALID_VALUE),
                         ((-4, 32, gf.GF_F16, 1, x.data_ptr(), q.data_ptr(), s.data_ptr()), gf.GF_ERR_INVALID_VALUE),
                         ((4, 32, gf.GF_BF16, 1, x, q, s), gf.GF_ERR_INVALID_VALUE),
                         ((4, 32, gf.GF_F16, 1, x, q, None), gf.GF_ERR_INVALID_VALUE),
                         ((4, 32, gf.GF_F16, 1, x.data_ptr() + 2, q, s), gf.GF_ERR_INVALID_VALUE)):
        with pytest.raises(gf.GfError) as err:
            gf.gf_fp8_quantize(*args)
        assert err.value.status == status
    gf.gf_fp8_quantize(0, 32, gf.GF_F16, 1, None, None, None)
    gf.gf_fp8_quantize(4, 0, gf.GF_F16, 1, None, None, None)


# ----------------------------------------------------------------- products
def operand(shape, seed):
    """e4m3 values over the type's range, zeros among them."""
    v = torch.randn(*shape, generator=gen(seed), device="cuda") * 24
    v = torch.where(torch.rand(*shape, generator=gen(seed + 100), device="cuda") < 0.1, 0.0, v)
    return v.to(torch.float8_e4m3fn)


def scales(shape, seed):
    """fp32 scales that no power of two is, some zero."""
    s = torch.exp2(torch.randn(*shape, generator=gen(seed), device="cuda") * 2) * 1e-3
    return torch.where(torch.rand(*shape, generator=gen(seed + 100), device="cuda") < 0.02, 0.0, s)


def values(q, s, block_rows):
    n, k = q.shape[-2:]
    wide = s.double().repeat_interleave(block_rows, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]
    return q.double() * wide


def split(m, groups, seed):
    """offsets of `groups` groups over m rows: empty ones, one row, the rest."""
    rng = np.random.default_rng(seed)
    cuts = np.sort(rng.integers(0, m + 1, groups - 1)) if groups > 1 else np.zeros(0, int)
    if groups > 3:
        cuts[0] = 0
        cuts[1] = min(1, m)
        cuts[2] = cuts[1]
    return np.concatenate([[0], np.sort(cuts), [m]])


def by_group(off, a, b):
    """rows of each group of a times its b^T, in 64 bits; zeros for rows of no group"""
    out = torch.zeros(a.shape[0], b.shape[1], dtype=torch.float64, device="cuda")
    for g in range(b.shape[0]):
        out[off[g]:off[g + 1]] = a[off[g]:off[g + 1]] @ b[g].t()
    return out


SHAPES = [  # m, n, k, groups
    (1, 8, 16, 1), (1, 136, 5120, 1), (3, 128, 128, 1), (16, 256, 384, 1), (17, 264, 272, 1), (64, 520, 1040, 1),
    (65, 128, 2048, 1), (200, 72, 144, 1), (300, 640, 512, 1), (1030, 1288, 656, 1), (2048, 1024, 1024, 1),
    (40, 256, 256, 5), (500, 136, 400, 7), (3000, 264, 272, 9), (1500, 384, 1040, 4), (700, 264, 128, 130), (33, 128, 256, 1024),
]


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("m,n,k,groups", SHAPES)
def test_matmul(m, n, k, groups, kernel):
    """|error| <= k 2^-23 sum |a b| (k additions, whatever their rounding, of
    products that are exact, and the scales' roundings) + the output's rounding."""
    dtype = gf.GF_BF16 if (m + n) % 3 else gf.GF_F16
    a, b = operand((m, k), 1), operand((groups, n, k), 2)
    sa, sb = scales((m, -(-k // 128)), 3), scales((groups, -(-n // 128), -(-k // 128)), 4)
    off = split(m, groups, 5)
    plan = gf.gf_fp8_matmul_plan(m, n, k, groups, dtype)
    gf.gf_plan_set_option(plan, gf.GF_OPT_KERNEL, kernel)
    out = torch.full((m, n), float("nan"), dtype=TDT[dtype], device="cuda")
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    gf.gf_fp8_matmul_execute(plan, a, sa, b, sb, offsets=None if groups == 1 else offsets, out=out)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    av, bv = values(a, sa, 1), values(b, sb, 128)
    want, mag = by_group(off, av, bv), by_group(off, av.abs(), bv.abs())
    u, tiny = ROUND[dtype]
    bound = (k + 4) * 2.0 ** -23 * mag
    bound = bound + u * (want.abs() + bound) + tiny
    diff = (out.double() - want).abs()
    assert bool((diff <= bound).all()), f"{(diff / (mag + 1e-300)).max().item():.3e} of sum |a b|"
    again = torch.empty_like(out)
    gf.gf_fp8_matmul_execute(plan, a, sa, b, sb, offsets=None if groups == 1 else offsets, out=again)
    assert torch.equal(out, again)
    assert gf.gf_plan_describe(plan)["launches"] == 1
    plan.free()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("m,n,k,groups", [
    (1, 16, 16, 1), (1, 400, 2048, 1), (17, 128, 272, 1), (65, 272, 512, 1), (300, 256, 1040, 3), (1000, 144, 256, 6),
    (600, 384, 384, 2), (70, 128, 256, 200)])
def test_swiglu_quant(m, n, k, groups, kernel):
    """e4m3 values times scales against h = silu(gate) up in 64 bits: half a
    step of e4m3 (2^-4 of the value, or 2^-10 scales below the type's normal
    range), at a scale that may be one power of two larger where the block's
    maximum lies at 448 times one, and h's own error: that of the products
    (as above, times the derivative of silu(g) u, at most 1.1 |u| and |g|)
    and 2^-20 of h for the exponential and the division."""
    a, b, b2 = operand((m, k), 11), operand((groups, n, k), 12), operand((groups, n, k), 13)
    kb, nb = -(-k // 128), -(-n // 128)
    sa = scales((m, kb), 14)
    sb, sb2 = scales((groups, nb, kb), 15), scales((groups, nb, kb), 16)
    off = split(m, groups, 17)
    if groups > 1:
        off[-1] = m - m // 10  # the last rows are no group's
        off = np.minimum(off, off[-1])
    plan = gf.gf_fp8_matmul_plan(m, n, k, groups, gf.GF_BF16, gf.GF_FP8_EPILOG_SWIGLU_QUANT)
    gf.gf_plan_set_option(plan, gf.GF_OPT_KERNEL, kernel)
    q = torch.full((m, n), 0x55, dtype=torch.uint8, device="cuda")
    qs = torch.full((m, nb), float("nan"), device="cuda")
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    gf.gf_fp8_matmul_execute(plan, a, sa, b, sb, b2, sb2, offsets, q, qs)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    av, gv, uv = values(a, sa, 1), values(b, sb, 128), values(b2, sb2, 128)
    g, u = by_group(off, av, gv), by_group(off, av, uv)
    eg = (k + 4) * 2.0 ** -23 * by_group(off, av.abs(), gv.abs())
    eu = (k + 4) * 2.0 ** -23 * by_group(off, av.abs(), uv.abs())
    h = g * torch.sigmoid(g) * u
    eh = 1.1 * u.abs() * eg + g.abs() * eu + 1.1 * eg * eu + 2.0 ** -20 * h.abs() + 1e-30
    pad = torch.nn.functional.pad(h, (0, -n % 128)).view(m, nb, 128).abs().amax(2)
    epad = torch.nn.functional.pad(eh, (0, -n % 128)).view(m, nb, 128).amax(2)
    lo, hi = quantized_scale(pad - epad), quantized_scale(pad + epad)
    got = qs.double()
    zero = pad <= epad  # the block's h may have rounded to zeros: scale 1 or a small one
    assert bool(((got >= lo) & (got <= hi) | zero).all())
    deq = q.view(torch.float8_e4m3fn).double() * got.repeat_interleave(128, 1)[:, :n]
    half = torch.maximum(2.0 ** -4 * (h.abs() + eh), 2.0 ** -10 * got.repeat_interleave(128, 1)[:, :n])
    ok = (deq - h).abs() <= half + eh
    wide_zero = zero.repeat_interleave(128, 1)[:, :n]
    assert bool((ok | (wide_zero & (deq.abs() <= 2 * eh + 1e-30))).all())
    assert bool((deq[off[-1]:] == 0).all()) and bool((qs[off[-1]:] == 1).all())
    plan.free()


def quantized_scale(top):
    """The smallest power of two s with top / s <= 448, 0 where top <= 0 (by numpy's exact ldexp)."""
    top = top.cpu().numpy()
    part, power = np.frexp(np.maximum(top, 0) / 448)
    power = np.maximum(np.where(part == 0.5, power - 1, power), -126)
    return torch.from_numpy(np.where(top <= 0, 0.0, np.ldexp(np.ones_like(top), power))).cuda()


def test_offsets_out_of_range_stay_inside():
    """Offsets that decrease or pass m: bounded by the kernel, no stray access;
    the rows of each group come out as for the bounded offsets."""
    m, n, k, groups = 300, 136, 144, 6
    raw = np.array([7, 50, 20, -5, 2 ** 31 - 1, 100, 90], np.int32)
    off = np.array([0, 50, 50, 50, 300, 300, 300])
    a, b = operand((m, k), 21), operand((groups, n, k), 22)
    sa, sb = scales((m, 2), 23), scales((groups, 2, 2), 24)
    for kernel in KERNELS:
        plan = gf.gf_fp8_matmul_plan(m, n, k, groups, gf.GF_BF16)
        gf.gf_plan_set_option(plan, gf.GF_OPT_KERNEL, kernel)
        flat = torch.full((m * n + 8192,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = flat[4096:4096 + m * n].view(m, n)
        gf.gf_fp8_matmul_execute(plan, a, sa, b, sb, offsets=torch.from_numpy(raw).cuda(), out=out)
        good = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        gf.gf_fp8_matmul_execute(plan, a, sa, b, sb, offsets=torch.from_numpy(off.astype(np.int32)).cuda(), out=good)
        assert torch.equal(out, good)
        assert bool((flat[:4096] == 7).all()) and bool((flat[-4096:] == 7).all())
        plan.free()


@pytest.mark.parametrize("kernel", KERNELS)
def test_every_tail_length(kernel):
    """Groups whose rows end on both sides of every tile size, and in more
    tiles than the grid has CTAs."""
    counts = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 384, 385, 511, 512, 513] * 3
    off = np.concatenate([[0], np.cumsum(counts)])
    m, groups, n, k = int(off[-1]), len(counts), 1416, 144
    plan = gf.gf_fp8_matmul_plan(m, n, k, groups, gf.GF_BF16)
    gf.gf_plan_set_option(plan, gf.GF_OPT_KERNEL, kernel)
    a, b = operand((m, k), 71), operand((groups, n, k), 72)
    sa, sb = scales((m, 2), 73), scales((groups, 12, 2), 74)
    out = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    gf.gf_fp8_matmul_execute(plan, a, sa, b, sb, offsets=torch.from_numpy(off.astype(np.int32)).cuda(), out=out)
    av, bv = values(a, sa, 1), values(b, sb, 128)
    want, mag = by_group(off, av, bv), by_group(off, av.abs(), bv.abs())
    bound = (k + 4) * 2.0 ** -23 * mag
    bound = bound + 2.0 ** -8 * (want.abs() + bound)
    assert bool(((out.double() - want).abs() <= bound).all())
    plan.free()


@pytest.mark.parametrize("kernel", KERNELS)
def test_nan_rows_stay_alone(kernel):
    """A NaN in one row (as a value, or as its scale) reaches that row's outputs only."""
    m, n, k = 100, 136, 272
    a, b = operand((m, k), 31), operand((1, n, k), 32)
    sa, sb = scales((m, 3), 33), scales((1, 2, 3), 34)
    plan = gf.gf_fp8_matmul_plan(m, n, k, 1, gf.GF_BF16)
    gf.gf_plan_set_option(plan, gf.GF_OPT_KERNEL, kernel)
    clean, out = (torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gf.gf_fp8_matmul_execute(plan, a, sa, b, sb, out=clean)
    a.view(torch.uint8)[40, 3] = 0x7F
    sa[70, 1] = float("nan")
    gf.gf_fp8_matmul_execute(plan, a, sa, b, sb, out=out)
    assert bool(out[40].isnan().all()) and bool(out[70].isnan().all())
    rest = [i for i in range(m) if i not in (40, 70)]
    assert torch.equal(out[rest], clean[rest])
    plan.free()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("m,n,k,groups", [(1, 16, 16, 1), (17, 144, 272, 3), (300, 272, 144, 4), (513, 400, 128, 2)])
def test_no_stray_stores(m, n, k, groups, kernel):
    """Outputs and scales between canaries, at sizes that end inside every tile."""
    kb, nb = -(-k // 128), -(-n // 128)
    a, b = operand((m, k), 91), operand((groups, n, k), 92)
    sa, sb = scales((m, kb), 93), scales((groups, nb, kb), 94)
    off = torch.from_numpy(split(m, groups, 95).astype(np.int32)).cuda()

    def between(count, dtype):
        flat = torch.full((8192 + count * torch.empty(0, dtype=dtype).element_size(),), 0x5A, dtype=torch.uint8, device="cuda")
        return flat, flat[4096:-4096].view(dtype)

    flats = []
    for quant in (False, True):
        epilog = gf.GF_FP8_EPILOG_SWIGLU_QUANT if quant else gf.GF_FP8_EPILOG_NONE
        plan = gf.gf_fp8_matmul_plan(m, n, k, groups, gf.GF_F16, epilog)
        gf.gf_plan_set_option(plan, gf.GF_OPT_KERNEL, kernel)
        flat, out = between(m * n, torch.uint8 if quant else torch.half)
        flat_s, os = between(m * nb, torch.float32)
        gf.gf_fp8_matmul_execute(plan, a, sa, b, sb, b if quant else None, sb if quant else None, off, out,
                                 os if quant else None)
        assert gf.gf_plan_status(plan) == gf.GF_OK
        flats += [flat, flat_s]
        plan.free()
    assert all(bool((f[:4096] == 0x5A).all()) and bool((f[-4096:] == 0x5A).all()) for f in flats)


@pytest.mark.parametrize("m,n,k,kernel", [
    (140000, 136, 16400, 3), (140000, 136, 16400, 4), (300000, 16384, 16, 3), (300000, 16384, 16, 4), (16, 16384, 140016, 1)])
def test_past_32_bit_offsets(m, n, k, kernel):
    """Operands and outputs of more than 2^31 bytes and elements: the first and
    the last rows, whose operands are set, come out right, the others are zero."""
    kb, nb = -(-k // 128), -(-n // 128)
    a = torch.zeros(m, k, dtype=torch.float8_e4m3fn, device="cuda")
    b = torch.zeros(1, n, k, dtype=torch.float8_e4m3fn, device="cuda")
    rows = [0, 1, m // 2, m - 2, m - 1] if m > 16 else list(range(m))
    cols = [0, n // 2, n - 1]
    a.view(torch.uint8)[rows] = operand((len(rows), k), 81).view(torch.uint8)
    b.view(torch.uint8)[0, cols] = operand((len(cols), k), 82).view(torch.uint8)
    sa, sb = torch.ones(m, kb, device="cuda"), scales((1, nb, kb), 83)
    sa[rows] = scales((len(rows), kb), 84)
    plan = gf.gf_fp8_matmul_plan(m, n, k, 1, gf.GF_BF16)
    gf.gf_plan_set_option(plan, gf.GF_OPT_KERNEL, kernel)
    out = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
    gf.gf_fp8_matmul_execute(plan, a, sa, b, sb, out=out)
    assert gf.gf_plan_status(plan) == gf.GF_OK
    av = values(a[rows], sa[rows], 1)
    bv = torch.stack([values(b[0, c:c + 1], sb[0, c // 128:c // 128 + 1], 1)[0] for c in cols])
    want, mag = av @ bv.t(), av.abs() @ bv.abs().t()
    bound = (k + 4) * 2.0 ** -23 * mag
    bound = bound + 2.0 ** -8 * (want.abs() + bound)
    assert bool(((out[rows][:, cols].double() - want).abs() <= bound).all())
    out[torch.tensor(rows)[:, None].cuda(), torch.tensor(cols).cuda()] = 0
    assert int(torch.count_nonzero(out)) == 0
    plan.free()


def test_empty():
    for m, n, k in ((0, 128, 128), (4, 0, 128)):
        plan = gf.gf_fp8_matmul_plan(m, n, k, 1, gf.GF_F16)
        gf.gf_fp8_matmul_execute(plan, None, None, None, None)
        assert gf.gf_plan_status(plan) == gf.GF_OK
        plan.free()
    plan = gf.gf_fp8_matmul_plan(5, 136, 0, 1, gf.GF_F16)  # k = 0: the product is zero
    out = torch.full((5, 136), float("nan"), dtype=torch.half, device="cuda")
    gf.gf_fp8_matmul_execute(plan, None, None, None, None, out=out)
    assert gf.gf_plan_status(plan) == gf.GF_OK and bool((out == 0).all())
    plan.free()


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("quant", [False, True])
def test_wait_limit_is_reported(kernel, quant):
    """A skipped stage load: the bounded waits give up, the status says so, and the plan works again after."""
    m, n, k = 300, 384, 2048
    a, b = operand((m, k), 41), operand((1, n, k), 42)
    sa, sb = scales((m, 16), 43), scales((1, 3, 16), 44)
    epilog = gf.GF_FP8_EPILOG_SWIGLU_QUANT if quant else gf.GF_FP8_EPILOG_NONE
    plan = gf.gf_fp8_matmul_plan(m, n, k, 1, gf.GF_BF16, epilog)
    gf.gf_plan_set_option(plan, gf.GF_OPT_KERNEL, kernel)
    gf.gf_plan_set_option(plan, gf.GF_OPT_WAIT_LIMIT_US, 5000)
    out = torch.zeros(m, n, dtype=torch.uint8 if quant else torch.bfloat16, device="cuda")
    os = torch.zeros(m, 3, device="cuda") if quant else None
    b2, sb2 = (b, sb) if quant else (None, None)

    def go():
        out.zero_()
        gf.gf_fp8_matmul_execute(plan, a, sa, b, sb, b2, sb2, out=out, out_scale=os)

    go()
    assert gf.gf_plan_status(plan) == gf.GF_OK
    first = out.clone()
    gf.gf_plan_set_option(plan, gf.GF_OPT_FAULT_DROP_LOAD, 3)
    go()
    assert gf.gf_plan_status(plan) == gf.GF_ERR_DEVICE_TIMEOUT
    gf.gf_plan_set_option(plan, gf.GF_OPT_FAULT_DROP_LOAD, 0)
    go()
    assert gf.gf_plan_status(plan) == gf.GF_OK
    assert torch.equal(out, first)
    plan.free()


def test_streams_and_graph():
    """Two plans on two streams at once, and a captured call replayed with other rows, give the same bits."""
    m, n, k, groups = 400, 264, 1040, 9
    a, b = operand((m, k), 51), operand((groups, n, k), 52)
    sa, sb = scales((m, 9), 53), scales((groups, 3, 9), 54)
    offsets = torch.from_numpy(split(m, groups, 55).astype(np.int32)).cuda()
    plans = [gf.gf_fp8_matmul_plan(m, n, k, groups, gf.GF_BF16) for _ in range(3)]
    outs = [torch.empty(m, n, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    for p, o, s in zip(plans, outs, (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream())):
        gf.gf_fp8_matmul_execute(p, a, sa, b, sb, offsets=offsets, out=o, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gf.gf_fp8_matmul_execute(plans[0], a, sa, b, sb, offsets=offsets, out=outs[0])
    a.copy_(operand((m, k), 56))
    offsets.copy_(torch.from_numpy(split(m, groups, 57).astype(np.int32)).cuda())
    graph.replay()
    gf.gf_fp8_matmul_execute(plans[1], a, sa, b, sb, offsets=offsets, out=outs[1])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])


def test_refusals():
    m, n, k = 16, 64, 128
    a, b = operand((m, k), 61), operand((1, n, k), 62)
    sa, sb = scales((m, 1), 63), scales((1, 1, 1), 64)
    out = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    plan = gf.gf_fp8_matmul_plan(m, n, k, 1, gf.GF_BF16)
    good = dict(A=a, a_scale=sa, B=b, b_scale=sb, out=out)
    for name, v in (("A", None), ("a_scale", None), ("B", None), ("b_scale", None), ("out", None),
                    ("A", a.t()), ("A", a.float()), ("a_scale", sa.half()), ("B", b[:, :8]), ("out", out.half()),
                    ("out", out.data_ptr() + 2), ("A", a.cpu())):
        with pytest.raises(gf.GfError) as err:
            gf.gf_fp8_matmul_execute(plan, **{**good, name: v})
        assert err.value.status == gf.GF_ERR_INVALID_VALUE
    grouped = gf.gf_fp8_matmul_plan(m, n, k, 2, gf.GF_BF16)
    b2, s2 = operand((2, n, k), 65), scales((2, 1, 1), 66)
    with pytest.raises(gf.GfError) as err:  # two groups need offsets
        gf.gf_fp8_matmul_execute(grouped, a, sa, b2, s2, out=out)
    assert err.value.status == gf.GF_ERR_INVALID_VALUE
    dual = gf.gf_fp8_matmul_plan(m, n, k, 1, gf.GF_BF16, gf.GF_FP8_EPILOG_SWIGLU_QUANT)
    q, qs = torch.zeros(m, n, dtype=torch.uint8, device="cuda"), torch.zeros(m, 1, device="cuda")
    for b2, s2, scale in ((None, sb, qs), (b, None, qs), (b, sb, None)):
        with pytest.raises(gf.GfError) as err:
            gf.gf_fp8_matmul_execute(dual, a, sa, b, sb, b2, s2, out=q, out_scale=scale)
        assert err.value.status == gf.GF_ERR_INVALID_VALUE
    for p in (plan, dual):
        for option, value, status in ((gf.GF_OPT_SPLIT_K, 2, gf.GF_ERR_UNSUPPORTED),
                                      (gf.GF_OPT_KERNEL, 99, gf.GF_ERR_INVALID_VALUE),
                                      (gf.GF_OPT_WAIT_LIMIT_US, 1, gf.GF_ERR_INVALID_VALUE),
                                      (77, 0, gf.GF_ERR_INVALID_VALUE)):
            with pytest.raises(gf.GfError) as err:
                gf.gf_plan_set_option(p, option, value)
            assert err.value.status == status
    with pytest.raises(gf.GfError):
        gf.gf_matmul_execute(plan, a, b, out=out)
    matmul = gf.gf_matmul_plan(64, 64, 64, gf.GF_BF16, gf.GF_EPILOG_NONE)
    with pytest.raises(gf.GfError):
        gf.gf_fp8_matmul_execute(matmul, **good)
    assert gf.lib().gf_fp8_matmul_execute(matmul.handle, *[a.data_ptr()] * 9, None) == gf.GF_ERR_INVALID_VALUE


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("m,n,k,groups", [
    (40, 256, 6400, 1), (100, 136, 5120, 3), (64, 264, 8192, 1), (128, 2600, 5120, 1), (500, 2600, 5120, 1), (9, 1000, 9872, 4)])
def test_split_tiles(m, n, k, groups, kernel):
    """Tiles whose k falls to several CTAs, some in the second round only, joined in k order."""
    test_matmul(m, n, k, groups, kernel)


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("m,n,k,groups", [(40, 272, 5120, 1), (30, 144, 4112, 3), (200, 1040, 2064, 2)])
def test_split_tiles_swiglu(m, n, k, groups, kernel):
    test_swiglu_quant(m, n, k, groups, kernel)


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("blocks", [7, 8, 9, 15, 16, 17, 24, 25])
def test_blocks_of_k(blocks, kernel):
    """Numbers of k-blocks around the groups that their scales come in, over several tiles of each CTA."""
    test_matmul(1500, 2056, 128 * blocks - 16, 3, kernel)
