"""The 4-bit linear at the ends of its ranges: row factors far from 1, weights without rows,
the longest rows.

Tolerance of a product as in the linear's own tests: half a BF16 step of the result (2^-8
relative; 2^-134 where the result is subnormal in BF16), and for the FP32 accumulation and the
factors 2^-22 a step of 64 products, and 8 steps more, of the sum of the magnitudes."""
import copy
import io

import pytest
import torch

import block_wise_w8a8_b200 as w8
import fp4_ref as ref

pytestmark = pytest.mark.gpu
FORMATS = ("mxfp4", "nvfp4")


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert w8.device_error() == 0


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _nvfp4(rows, K, factor, seed, zero=False):
    """An nvfp4 matrix with these row factors (a number or a row's each)."""
    g = _gen(seed)
    codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, generator=g) * (0 if zero else 1)
    s = torch.randint(40, 100, (rows, K // 16), generator=g).to(torch.uint8)
    f = torch.full((rows,), factor) if isinstance(factor, float) else factor
    return w8.FP4Tensor(codes.to(torch.uint8).cuda(), w8.fp4_tile_scales(s).cuda(), f.float().cuda(), "nvfp4")


def _check(y, x, w, bias):
    xv, wv = ref.tensor_values(x), ref.tensor_values(w)
    b = 0.0 if bias is None else bias.double()
    want, size = xv @ wv.T + b, xv.abs() @ wv.abs().T + abs(b)
    tol = want.abs() * 2.0 ** -8 + size * (x.K / 64 + 8) * 2.0 ** -22 + 2.0 ** -134
    # a result that rounds past the largest BF16 number (2^128 - 2^119 from half a step above
    # it on) is an infinity; within the tolerance of that border either is right
    y, border = y.double(), 2.0 ** 128 - 2.0 ** 119
    big = y.isinf() & (y.sign() == want.sign()) & (want.abs() + tol >= border)
    bad = (~((y - want).abs() <= tol) & ~big).nonzero()
    assert not len(bad), (f"{len(bad)} of {y.numel()} off, first {bad[0].tolist()}: {y[tuple(bad[0])].item()} "
                          f"for {want[tuple(bad[0])].item()}")


# few tokens (K split and not), pairs of CTAs with and without TMA stores, half tiles
SHAPES = [(3, 512, 264), (3, 4096, 100), (40, 512, 264), (300, 512, 264), (300, 512, 263), (700, 96, 1000)]


@pytest.mark.parametrize("M,K,N", [(1, 16384, 33 * 128), (1, 16384, 34 * 128), (37, 16384, 36 * 128), (1, 4096, 71 * 128), (1, 4096, 72 * 128),
                                   (20, 4096, 72 * 128), (3, 2048, 148 * 128), (3, 2048, 149 * 128), (768, 16384, 768), (1664, 37120, 1408),
                                   (1664, 40960, 1536)])
def test_sizes_around_the_limits_of_splitting(M, K, N):
    """Numbers of tiles on both sides of those that clusters of 8, 4 and 2 take at once, and of
    the one from which pairs of CTAs take long rows."""
    x, w = _nvfp4(M, K, 1.4, 1), _nvfp4(N, K, 1.7, 2)
    bias = torch.randn((N,), generator=_gen(3)).bfloat16().cuda()
    y = w8.fp4_linear_prequant(x, w8.FP4Weight(q=w), bias)
    _check(y, x, w, bias)
    assert torch.equal(w8.fp4_linear_prequant(x, w8.FP4Weight(q=w), bias), y)


# exponents of x's and w's factors.  The quantizer's own lie between 2^-111.4 and 2^116.6.  The
# products of the first five pairs leave FP32's normal range, the sums times both do not.
@pytest.mark.parametrize("ex,ew", [(-101, -41), (-41, -101), (-111, -20), (-70, -70), (115, 2), (100, -100), (-111, 116), (116, -111),
                                   (0, 0), (60, 50)])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_factors_far_from_one(M, K, N, ex, ew):
    x, w = _nvfp4(M, K, 1.4 * 2.0 ** ex, 1), _nvfp4(N, K, 1.7 * 2.0 ** ew, 2)
    wt = w8.FP4Weight(q=w)
    bias = (torch.randn((N,), generator=_gen(3)) * 2.0 ** max(ex + ew, -120)).bfloat16().cuda()
    for b in (None, bias):
        _check(w8.fp4_linear_prequant(x, wt, b), x, w, b)


@pytest.mark.parametrize("ex,ew", [(100, 60), (116, 116), (127, 1), (-111, -111)])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_a_zero_sum_is_the_bias(M, K, N, ex, ew):
    """Whatever the factors, also where their product is no FP32 number."""
    x, w = _nvfp4(M, K, 1.4 * 2.0 ** ex, 1, zero=True), _nvfp4(N, K, 1.7 * 2.0 ** ew, 2)
    wt = w8.FP4Weight(q=w)
    bias = torch.randn((N,), generator=_gen(3)).bfloat16().cuda()
    assert bool((w8.fp4_linear_prequant(x, wt, bias) == bias).all())
    assert bool((w8.fp4_linear_prequant(x, wt) == 0).all())


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_rows_of_every_size_in_one_tile(M, K, N):
    """Factors of every size next to one another, NaN among them: each row and column is right,
    and a row has the bits that it has among rows like itself."""
    ex = torch.tensor([-111, -70, -20, 0, 20, 90])[torch.randint(0, 6, (M,), generator=_gen(4))].double()
    ew = torch.tensor([-111, -60, -10, 0, 10, 30])[torch.randint(0, 6, (N,), generator=_gen(5))].double()
    x, w = _nvfp4(M, K, 1.3 * torch.exp2(ex), 6), _nvfp4(N, K, 1.6 * torch.exp2(ew), 7)
    y = w8.fp4_linear_prequant(x, w8.FP4Weight(q=w))
    _check(y, x, w, None)
    ones = x.factor.clone()
    ones[ex != 0] = 1.3
    like = w8.fp4_linear_prequant(w8.FP4Tensor(x.codes, x.scales, ones, "nvfp4"), w8.FP4Weight(q=w))
    assert torch.equal(like[(ex == 0).cuda()].view(torch.int16), y[(ex == 0).cuda()].view(torch.int16))
    bad = x.factor.clone()
    bad[M // 2] = float("nan")
    z = w8.fp4_linear_prequant(w8.FP4Tensor(x.codes, x.scales, bad, "nvfp4"), w8.FP4Weight(q=w))
    rest = torch.arange(M) != M // 2
    assert bool(z[M // 2].isnan().all()) and torch.equal(z[rest].view(torch.int16), y[rest].view(torch.int16))


@pytest.mark.parametrize("ex,ew", [(-90, -30), (-30, -90), (100, -60), (100, 60)])
@pytest.mark.parametrize("M", [1, 4, 20, 300])
def test_linear_of_rows_far_from_one(M, ex, ew):
    """The same from BF16 rows, quantized inside the product and before it; one row of zeros."""
    K, N = 992, 264
    x = (torch.randn((M, K), generator=_gen(M)) * 2.0 ** ex).bfloat16()
    x[M - 1] = 0
    w = w8.FP4Weight((torch.randn((N, K), generator=_gen(1)) * 2.0 ** ew).bfloat16().cuda(), keep_bf16=False)
    y = w8.fp4_linear(x.cuda(), w)
    _check(y, w8.fp4_quantize(x.cuda()), w.q, None)
    assert bool((y[M - 1] == 0).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [40, 64])
def test_a_weight_without_rows(fmt, K):
    w = torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    for M in (0, 1, 7):
        x = torch.randn((M, K), generator=_gen(M)).bfloat16().cuda()
        y, path = w8.fp4_linear(x, w8.FP4Weight(w, fmt), return_path=True)
        assert y.shape == (M, 0) and path == w8.PATH_NONE
        if K == 64:
            q = w8.fp4_quantize(w, fmt)
            given = w8.FP4Tensor(q.codes, q.scales, q.factor, fmt)
            for wt in (w8.FP4Weight(w, fmt, keep_bf16=False), w8.FP4Weight(q=q), w8.FP4Weight(q=given)):
                assert w8.fp4_linear(x, wt).shape == (M, 0)
                assert w8.fp4_linear_prequant(w8.fp4_quantize(x, fmt), wt).shape == (M, 0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("given", [False, True])
def test_copies_stand_for_their_own_tensors(fmt, given):
    """A deep copy, and one from a file, keep their values when the first matrix is written
    again or gone; a shallow copy is another name for it."""
    def save(q):
        f = io.BytesIO()
        torch.save(q, f)
        f.seek(0)
        return torch.load(f, weights_only=False)
    x, other = (torch.randn((130, 96), generator=_gen(s)).bfloat16().cuda() for s in (1, 2))
    q = w8.fp4_quantize(x, fmt)
    if given:
        q = w8.FP4Tensor(q.codes.clone(), q.scales.clone(), None if q.factor is None else q.factor.clone(), fmt)
    want = w8.fp4_dequantize(q)
    deep, loaded, name = copy.deepcopy(q), save(q), copy.copy(q)
    w8.fp4_quantize(other, fmt, out=q)
    new = w8.fp4_dequantize(q)
    assert not torch.equal(new, want)
    del q
    for c, y in ((deep, want), (loaded, want), (name, new)):
        assert torch.equal(w8.fp4_dequantize(c), y)
        code = ref.values(ref.unpack(c.codes), ref.plain_scales(c), c.factor, fmt)
        assert torch.equal(code.float().bfloat16().double(), y.double())
        w = w8.FP4Weight(q=c)
        assert torch.equal(w8.fp4_linear_prequant(c, w), w8.fp4_linear_prequant(w8.fp4_quantize(x if y is want else other, fmt), w))


def test_rows_longer_than_the_formats_take():
    """The guard's BF16 path: no codes are made, and the results are the BF16 linear's."""
    K = 2 ** 24 + 32
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn((3, K), generator=g, device="cuda").bfloat16()
    wt = w8.FP4Weight(w, keep_bf16=False)
    assert wt.q is None and wt.w is w
    for M in (2, 7):
        x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
        y, path = w8.fp4_linear(x, wt, return_path=True)
        assert path == w8.PATH_BF16 and torch.equal(y, w8.bf16_linear(x, w))
    with pytest.raises(w8.W8A8Error) as e:
        w8.fp4_quantize(w)
    assert e.value.code == 2
