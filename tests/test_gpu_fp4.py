"""The microscaled 4-bit quantizer and linear on the GPU, through the binding and the C ABI,
against the 64-bit reference.

Codes (but for the sign of an nvfp4 zero, which the format's definition here leaves open),
scales and factors must equal the reference's bit for bit, and dequantized values the
reference's values rounded through FP32 to BF16.  Products are compared with the 64-bit
product of the values the codes stand for.  Their tolerance: half a BF16 step of the result
(2^-8 relative), plus the FP32 accumulation.  One step of the tensor cores adds 64 products
to the running sum; a step's error is a few units of FP32 in the last place of the largest
number involved, which the sum S of the magnitudes bounds: 2^-22 S a step, and 8 steps'
worth for the join of split sums, the factors and the bias."""
import ctypes
import os
import subprocess
import sys

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


def _rows(M, K, seed):
    """Heavy-tailed rows of very different sizes; from a few rows on also zero rows, zero
    blocks, subnormals, the largest finite values, and many exact ties."""
    g = _gen(seed)
    x = torch.randn((M, K), generator=g) / torch.rand((M, K), generator=g).clamp(min=1e-3).sqrt()
    x *= torch.exp(torch.rand((M, 1), generator=g) * 24 - 12)
    x = x.bfloat16()
    if M >= 8:
        x[0] = 0
        x[1] = torch.randint(-28, 29, (K,), generator=g) / 4            # quarters: ties
        x[2, : K // 2] = 0
        x[3] = (x[3].float() * 2.0 ** -126).bfloat16()                  # subnormals and zeros
        x[4] = torch.where(torch.rand((K,), generator=g) < 0.5, 3.3895e38, -1e38).bfloat16()
        x[5] = (torch.randn((K,), generator=g) * torch.exp(torch.rand((K,), generator=g) * -30)).bfloat16()
        x[6] = (2.0 ** -torch.randint(0, 40, (K,), generator=g).float()).bfloat16()
        x[7] = (torch.randn((K,), generator=g) * 2.0 ** -105).bfloat16()   # below the factor's floor
    return x


def _check_quantized(q, x, what):
    code, scales, factor = ref.quantize(x, q.format)
    assert torch.equal(ref.plain_scales(q).cpu(), scales), f"{what}: scales"
    got, want = q.codes.cpu(), ref.pack(code)
    if q.format == "nvfp4":
        got, want = ref.no_minus_zero(got), ref.no_minus_zero(want)
    bad = (got != want).nonzero()
    assert not len(bad), f"{what}: {len(bad)} code bytes differ, first at {bad[0].tolist()}"
    if factor is not None:
        assert torch.equal(q.factor.cpu().view(torch.int32)[~factor.isnan()], factor.view(torch.int32)[~factor.isnan()])
        assert torch.equal(q.factor.cpu().isnan(), factor.isnan())
    nb = x.shape[1] // ref.BLOCK[q.format]
    live = torch.zeros_like(q.scales)
    r = torch.arange(x.shape[0], device=live.device)[:, None]
    b = torch.arange(nb, device=live.device)[None, :]
    live[r // 128, b // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4] = 1
    assert not bool(q.scales[live == 0].any()), f"{what}: scales past the end"


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(1, 32), (2, 64), (9, 96), (33, 160), (129, 512), (8, 544), (300, 1056), (37, 4096),
                                 (8, 16384), (11, 16416), (8, 40000), (1300, 2080)])
def test_quantize_bit_exact(fmt, M, K):
    x = _rows(M, K, M * 7 + K)
    q = w8.fp4_quantize(x.cuda(), fmt)
    _check_quantized(q, x, f"{fmt} {M}x{K}")
    v = ref.values(ref.unpack(q.codes.cpu()), ref.plain_scales(q).cpu(), None, fmt, with_factor=False)
    v = v.float() if q.factor is None else v.float() * q.factor.cpu()[:, None]
    y = w8.fp4_dequantize(q).cpu()
    assert torch.equal(y.view(torch.int16), v.bfloat16().view(torch.int16))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K", [(9500, 992), (4800, 1504), (2500, 2560), (2400, 4096), (1900, 5120), (1600, 6144),
                                 (1200, 8192), (950, 10240), (790, 12256), (640, 16384)])
def test_quantize_many_rows(fmt, M, K):
    """Several rows a CTA: the first 41 against the plain form, the others their repetitions."""
    part = _rows(41, K, M + K)
    x = part.repeat(-(-M // 41), 1)[:M].contiguous()
    q, few = w8.fp4_quantize(x.cuda(), fmt), w8.fp4_quantize(part.cuda(), fmt)
    _check_quantized(few, part, f"{fmt} 41x{K}")
    again = torch.arange(M, device="cuda") % 41
    assert torch.equal(q.codes, few.codes[again])
    assert torch.equal(ref.plain_scales(q), ref.plain_scales(few)[again])
    if q.factor is not None:
        assert torch.equal(q.factor.view(torch.int32), few.factor.view(torch.int32)[again])


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_ties_and_near_ties(fmt):
    """Every BF16 significand against every other, over the binades that a block can hold:
    the rounding boundaries of codes and scales and their neighbours."""
    m = torch.arange(128, 256, dtype=torch.float32)
    K = 128 * ref.BLOCK[fmt]
    x = torch.zeros((128, 128, ref.BLOCK[fmt]))
    x[:, :, 0] = m[:, None] / 128                          # the block's largest
    e = torch.arange(1, ref.BLOCK[fmt])
    x[:, :, 1:] = m[None, :, None] / 256 / 2.0 ** (e % 6)[None, None, :]
    x[:, :, 1:] *= torch.where(e % 2 == 0, -1.0, 1.0)
    x = x.view(128, K).bfloat16()
    _check_quantized(w8.fp4_quantize(x.cuda(), fmt), x, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_quantize_infinities_and_nan(fmt, value):
    x = torch.randn((5, 96), generator=_gen(3)).bfloat16()
    x[2, 40] = value
    q = w8.fp4_quantize(x.cuda(), fmt)
    _check_quantized(q, x, fmt)
    y = w8.fp4_dequantize(q)
    hit = torch.zeros((5, 96), dtype=torch.bool)
    hit[2, 32:64] = True
    if fmt == "nvfp4":
        hit[2] = True
    assert torch.equal(y.isnan().cpu(), hit)
    out = w8.fp4_linear(x.cuda(), w8.FP4Weight(torch.randn((7, 96), generator=_gen(4)).bfloat16().cuda(), fmt))
    assert bool(out[2].isnan().all()) and not bool(out[[0, 1, 3, 4]].isnan().any())


def _random_weight(N, K, fmt, seed, wide=False):
    """A weight given as codes: every code, and scales over their ordinary range (wide: from
    the smallest to the largest that keep the products finite)."""
    g = _gen(seed)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=g)
    nb = K // ref.BLOCK[fmt]
    if fmt == "mxfp4":
        s = torch.randint(90 if wide else 118, 160 if wide else 128, (N, nb), generator=g)
        factor = None
    else:
        s = torch.randint(0 if wide else 40, 127 if wide else 100, (N, nb), generator=g)
        factor = (torch.rand((N,), generator=g) + 0.5) * 2.0 ** -6
    return w8.FP4Tensor(codes.cuda(), w8.fp4_tile_scales(s.to(torch.uint8)).cuda(),
                        None if factor is None else factor.cuda(), fmt)


def _check_product(y, xq, wq, bias, what):
    xv, wv = ref.tensor_values(xq), ref.tensor_values(wq)
    want = xv @ wv.T
    size = xv.abs() @ wv.abs().T
    if bias is not None:
        want = want + bias.double()
        size = size + bias.double().abs()
    tol = want.abs() * 2.0 ** -8 + size * (xq.K / 64 + 8) * 2.0 ** -22
    err = (y.double() - want).abs()
    bad = (~(err <= tol)).nonzero()
    assert not len(bad), (f"{what}: {len(bad)} of {y.numel()} off, first {bad[0].tolist()}: "
                          f"{y[tuple(bad[0])].item()} for {want[tuple(bad[0])].item()}")


SHAPES = [(1, 32, 1), (1, 64, 130), (5, 96, 128), (16, 256, 256), (17, 288, 100), (31, 544, 257), (33, 1024, 129),
          (64, 2048, 384), (65, 160, 40), (100, 4096, 200), (128, 512, 512), (3, 8192, 24), (3, 131104, 40),
          (70, 262176, 9)]
LARGE = [(129, 64, 8), (129, 32, 1), (256, 256, 256), (257, 288, 255), (300, 544, 520), (512, 1056, 1000),
         (1000, 2048, 777), (640, 4096, 2056), (2100, 320, 3000),
         (1000, 16384, 8), (300, 8192, 1001), (70, 2048, 300), (19000, 96, 264), (2000, 70016, 264)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_product_few_tokens(fmt, M, K, N):
    _product_case(fmt, M, K, N)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K,N", LARGE)
def test_product_many_tokens(fmt, M, K, N):
    _product_case(fmt, M, K, N)


def _product_case(fmt, M, K, N):
    """Codes, scales and factors that differ in every row and block, a bias, and output rows
    behind the last one, which stay as they were; the same bits twice."""
    x = _random_weight(M, K, fmt, M + K)
    w = _random_weight(N, K, fmt, N + 2 * K, wide=fmt == "nvfp4")
    bias = torch.randn((N,), generator=_gen(N)).bfloat16().cuda() if (M + N) % 2 else None
    big = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    wt = w8.FP4Weight(q=w)
    y = w8.fp4_linear_prequant(x, wt, bias, out=big[:M])
    _check_product(y, x, w, bias, f"{fmt} {M}x{K}x{N}")
    assert bool((big[M:] == 7).all())
    assert torch.equal(w8.fp4_linear_prequant(x, wt, bias).view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("fmt", FORMATS)
def test_wide_power_of_two_scales(fmt):
    """Scales from the smallest kinds to large ones in one product."""
    x, w = _random_weight(40, 512, fmt, 1, wide=True), _random_weight(300, 512, fmt, 2, wide=True)
    _check_product(w8.fp4_linear_prequant(x, w8.FP4Weight(q=w)), x, w, None, fmt)
    x = _random_weight(400, 512, fmt, 3, wide=True)
    _check_product(w8.fp4_linear_prequant(x, w8.FP4Weight(q=w)), x, w, None, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M", [1, 20, 200, 1000])
def test_linear_is_quantize_and_product(fmt, M):
    K, N = 992, 264
    g = _gen(M)
    x = torch.randn((M, K), generator=g).bfloat16().cuda()
    w = (torch.randn((N, K), generator=g) * K ** -0.5).bfloat16().cuda()
    b = torch.randn((N,), generator=g).bfloat16().cuda()
    wt = w8.FP4Weight(w, fmt, keep_bf16=False)
    assert wt.w is None
    y, path = w8.fp4_linear(x, wt, b, return_path=True)
    assert path == w8.PATH_FP4
    xq = w8.fp4_quantize(x, fmt)
    assert torch.equal(y.view(torch.int16), w8.fp4_linear_prequant(xq, wt, b).view(torch.int16))
    _check_product(y, xq, wt.q, b, f"{fmt} {M}")
    y3 = w8.fp4_linear(x.view(1, M, K), wt, b, workspace=torch.empty(
        w8.fp4_linear_workspace_bytes(M, K, fmt), dtype=torch.uint8, device="cuda"))
    assert y3.shape == (1, M, N) and torch.equal(y3[0].view(torch.int16), y.view(torch.int16))
    # 4-bit quantization keeps a normal x and w to about 13% of the exact product
    exact = x.double() @ w.double().T + b.double()
    assert float((y.double() - exact).norm() / exact.norm()) < 0.2


def test_large_product_on_sampled_rows():
    """The benchmark's up-projection: rows from every part against the 64-bit product."""
    M, K, N = 16384, 4096, 16384
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    w = (torch.randn((N, K), generator=g, device="cuda") / 64).bfloat16()
    for fmt in FORMATS:
        wt = w8.FP4Weight(w, fmt)
        xq = w8.fp4_quantize(x, fmt)
        y = w8.fp4_linear_prequant(xq, wt)
        rows = torch.randint(0, M, (300,), generator=g, device="cuda")
        xv = ref.values(ref.unpack(xq.codes[rows]), ref.plain_scales(xq)[rows],
                        None if xq.factor is None else xq.factor[rows], fmt)
        wv = ref.tensor_values(wt.q)
        want, size = xv @ wv.T, xv.abs() @ wv.abs().T
        err = (y[rows].double() - want).abs()
        assert bool((err <= want.abs() * 2.0 ** -8 + size * (K / 64 + 8) * 2.0 ** -22).all()), fmt


@pytest.mark.parametrize("fmt", FORMATS)
def test_offsets_past_32_bits(fmt):
    """More than 2^31 elements of x and of y: the last rows are those of a call of their own."""
    M, K = 280000, 8192
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((256, K), generator=g, device="cuda").bfloat16().repeat((M + 255) // 256, 1)[:M].contiguous()
    x[-300:] = torch.randn((300, K), generator=g, device="cuda").bfloat16()
    q = w8.fp4_quantize(x, fmt)
    y = w8.fp4_dequantize(q)
    one = w8.fp4_quantize(x[-300:].contiguous(), fmt)
    assert torch.equal(q.codes[-300:], one.codes)
    assert torch.equal(ref.plain_scales(q)[-300:], ref.plain_scales(one))
    assert torch.equal(y[-300:].view(torch.int16), w8.fp4_dequantize(one).view(torch.int16))
    del x, y, q
    M, K = 70000, 256
    for N in (40000, 39999):
        x = _random_weight(M, K, fmt, 7)
        w = _random_weight(N, K, fmt, 8)
        y = w8.fp4_linear_prequant(x, w8.FP4Weight(q=w))
        assert y.numel() > 2 ** 31
        rows = torch.tensor([0, 1, 53687, 53688, M - 257, M - 1], device="cuda")
        xv = ref.tensor_values(x)[rows]
        wv = ref.tensor_values(w)
        want, size = xv @ wv.T, xv.abs() @ wv.abs().T
        err = (y[rows].double() - want).abs()
        assert bool((err <= want.abs() * 2.0 ** -8 + size * (K / 64 + 8) * 2.0 ** -22).all()), N
        del y


@pytest.mark.parametrize("fmt", FORMATS)
def test_output_at_any_even_address(fmt):
    """An output that starts two bytes past a 16-byte boundary, and a bias and factors that
    start anywhere their type may: the same bits as aligned ones."""
    for M, K, N in [(5, 256, 264), (300, 288, 520)]:
        x, w = _random_weight(M, K, fmt, 1), _random_weight(N, K, fmt, 2)
        bias = torch.randn((N + 1,), generator=_gen(3)).bfloat16().cuda()
        want = w8.fp4_linear_prequant(x, w8.FP4Weight(q=w), bias[1:].clone())
        flat = torch.full((M * N + 9,), 3.0, dtype=torch.bfloat16, device="cuda")
        out = flat[1:1 + M * N].view(M, N)
        if fmt == "nvfp4":
            big = torch.zeros((N + 1,), device="cuda")
            big[1:] = w.factor
            w = w8.FP4Tensor(w.codes, w.scales, big[1:], fmt)
        w8.fp4_linear_prequant(x, w8.FP4Weight(q=w), bias[1:], out=out)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        assert float(flat[0]) == 3 and bool((flat[1 + M * N:] == 3).all())


def test_one_dimension_and_empty_leading():
    wt = w8.FP4Weight(torch.randn((40, 96), generator=_gen(1)).bfloat16().cuda())
    x = torch.randn((3, 96), generator=_gen(2)).bfloat16().cuda()
    y = w8.fp4_linear(x, wt)
    assert torch.equal(w8.fp4_linear(x[1], wt).view(torch.int16), w8.fp4_linear(x[1:2], wt)[0].view(torch.int16))
    assert w8.fp4_linear(x.view(1, 3, 1, 96), wt).shape == (1, 3, 1, 40) and y.shape == (3, 40)


@pytest.mark.parametrize("fmt", FORMATS)
def test_few_rows_quantized_in_the_product(fmt):
    """1 to 5 rows on both sides of the quantizing product's limit, K from one block pair to
    several splits, rows of zeros and of very different sizes: the bits of the two calls."""
    for K, N in [(32, 1), (96, 130), (288, 100), (2080, 520), (4096, 4096), (16416, 136)]:
        w = w8.FP4Weight((torch.randn((N, K), generator=_gen(K)) * K ** -0.5).bfloat16().cuda(), fmt, keep_bf16=False)
        b = torch.randn((N,), generator=_gen(N)).bfloat16().cuda()
        x = (torch.randn((5, K), generator=_gen(5)) * torch.tensor([1, 300, 1e-4, 0, 7])[:, None]).bfloat16().cuda()
        for M in range(1, 6):
            y = w8.fp4_linear(x[:M], w, b)
            want = w8.fp4_linear_prequant(w8.fp4_quantize(x[:M], fmt), w, b)
            assert torch.equal(y.view(torch.int16), want.view(torch.int16)), (K, N, M)


def test_two_streams_at_once():
    """Calls of every kernel in flight on two streams: the bits of the calls one by one."""
    g = _gen(12)
    wt = [w8.FP4Weight((torch.randn((768, 1024), generator=g) / 32).bfloat16().cuda(), f) for f in FORMATS]
    xs = [torch.randn((M, 1024), generator=g).bfloat16().cuda() for M in (1, 3, 20, 100, 900)]
    want = [[w8.fp4_linear(x, w) for x in xs] for w in wt]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k] = [w8.fp4_linear(x, wt[k]) for x in xs]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(u.view(torch.int16), v.view(torch.int16)) for u, v in zip(a, b))


@pytest.mark.parametrize("M,K,N", [(3, 40, 16), (70, 1000, 65), (4, 0, 9)])
def test_guard_takes_bf16(M, K, N):
    g = _gen(K)
    x = torch.randn((M, K), generator=g).bfloat16().cuda()
    w = torch.randn((N, K), generator=g).bfloat16().cuda()
    b = torch.randn((N,), generator=g).bfloat16().cuda()
    y, path = w8.fp4_linear(x, w8.FP4Weight(w), b, return_path=True)
    assert path == w8.PATH_BF16
    assert torch.equal(y.view(torch.int16), w8.bf16_linear(x, w, b).view(torch.int16))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("M,K,N", [(1, 4096, 512), (5, 2048, 4096), (200, 1024, 1000)])
def test_weight_written_just_before_its_product(fmt, M, K, N):
    """The weight quantized again in place between products, eager and replayed: every product
    sees the codes of the call before it."""
    g = _gen(M + N)
    x = torch.randn((M, K), generator=g).bfloat16().cuda()
    ws = [torch.randn((N, K), generator=g).bfloat16().cuda() for _ in range(3)]
    want = [w8.fp4_linear(x, w8.FP4Weight(w, fmt)) for w in ws]
    q = w8.fp4_quantize(ws[0], fmt)
    wt = w8.FP4Weight(q=q)

    def run():
        out = []
        for w in ws * 4:
            w8.fp4_quantize(w, fmt, out=q)
            out.append(w8.fp4_linear(x, wt))
        return out
    torch.cuda.synchronize()
    for got in (run(), run()):
        assert all(torch.equal(a, b) for a, b in zip(got, want * 4))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want * 4))
        for y in got:
            y.zero_()


def test_empty():
    wt = w8.FP4Weight(torch.randn((8, 64), generator=_gen(1)).bfloat16().cuda())
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    y, path = w8.fp4_linear(x, wt, return_path=True)
    assert y.shape == (0, 8) and path == w8.PATH_NONE
    q = w8.fp4_quantize(x)
    assert q.codes.shape == (0, 32) and w8.fp4_dequantize(q).shape == (0, 64)
    assert w8.fp4_linear_prequant(q, wt).shape == (0, 8)


def test_rows_do_not_depend_on_the_batch():
    x = _rows(300, 2080, 11).cuda()
    for fmt in FORMATS:
        q = w8.fp4_quantize(x, fmt)
        for r in (0, 5, 128, 299):
            one = w8.fp4_quantize(x[r:r + 1].clone(), fmt)
            assert torch.equal(one.codes[0], q.codes[r])
            assert torch.equal(ref.plain_scales(one)[0], ref.plain_scales(q)[r])


def test_graph_capture_and_side_stream():
    K, N = 1024, 640
    wt = w8.FP4Weight((torch.randn((N, K), generator=_gen(1)) / 32).bfloat16().cuda())
    for M in (1, 48, 700):
        x = torch.randn((M, K), generator=_gen(M)).bfloat16().cuda()
        want = w8.fp4_linear(x, wt)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y = w8.fp4_linear(x, wt)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))
        graph = torch.cuda.CUDAGraph()
        static = x.clone()
        with torch.cuda.graph(graph):
            out = w8.fp4_linear(static, wt)
        for shift in (0, 1):
            static.copy_(x.roll(shift, 0))
            graph.replay()
            assert torch.equal(out.view(torch.int16), want.roll(shift, 0).view(torch.int16))


def test_first_call_inside_a_capture():
    """A process whose first call of each kernel is captured: the graph replays the bits of
    the eager calls that follow."""
    code = """
import torch, block_wise_w8a8_b200 as w8
g = torch.Generator().manual_seed(1)
x = [torch.randn((M, 1024), generator=g).bfloat16().cuda() for M in (2, 40, 700, 9000)]
w = torch.randn((520, 1024), generator=g).bfloat16().cuda()
torch.cuda.synchronize()
def run():
    wt = w8.FP4Weight(w)
    return [w8.fp4_linear(a, wt) for a in x] + list(w8.block_norm(x[3], x[3])) + [w8.block_norm_fp4(x[3], x[3])[1].codes]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(out, run()))
assert w8.device_error() == 0
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_c_abi_refusals():
    L = w8.lib()
    st = w8._stream(torch.device("cuda"))
    x = torch.zeros((64, 64), dtype=torch.bfloat16, device="cuda")
    q = w8.fp4_quantize(x)
    P = lambda t: t.data_ptr()  # noqa: E731
    quant = L.w8a8_fp4_quantize
    args = (64, 64, 1, P(q.codes), P(q.scales), P(q.factor), st)
    assert quant(P(x), *args) == 0
    assert quant(P(x), 64, 48, *args[2:]) == 2
    assert quant(P(x), 64, 0, *args[2:]) == 2
    assert quant(P(x), -1, 64, *args[2:]) == 1
    assert quant(P(x), 64, 64, 2, *args[3:]) == 1
    assert quant(P(x) + 2, *args) == 4
    assert quant(torch.zeros(8192).data_ptr(), *args) == 3
    assert quant(P(x), 64, 64, 0, P(q.codes), P(q.scales), P(q.factor), st) == 1    # MX has no factor
    assert quant(P(x), 64, 64, 1, P(q.codes), P(q.scales), None, st) == 1
    assert quant(P(x), 64, 64, 1, P(q.codes) + 8, P(q.scales), P(q.factor), st) == 4
    wt = w8.FP4Weight(x)
    y = torch.empty((64, 64), dtype=torch.bfloat16, device="cuda")
    path = ctypes.c_int()
    ws = torch.empty(w8.fp4_linear_workspace_bytes(64, 64), dtype=torch.uint8, device="cuda")
    lin = lambda K, rec, wsp, n: L.w8a8_fp4_linear(P(x), 64, K, rec, None, P(y), wsp, n, ctypes.byref(path), st)  # noqa: E731
    assert lin(64, wt.record(), P(ws), ws.numel()) == 0 and path.value == w8.PATH_FP4
    assert lin(64, wt.record(), P(ws), ws.numel() - 1) == 5
    assert lin(64, wt.record(), None, 0) == 5
    assert lin(32, wt.record(), P(ws), ws.numel()) == 1                              # another K than the weight's
    none = w8._FP4Weight(64, 40, 1, 0, P(q.codes), P(q.scales), P(q.factor))
    assert lin(40, ctypes.byref(none), P(ws), ws.numel()) == 2                       # no BF16 copy to fall back on
    with pytest.raises(w8.W8A8Error):
        w8.fp4_linear(x, wt, workspace=ws[:-1])
    with pytest.raises(ValueError):
        w8.fp4_linear_prequant(w8.fp4_quantize(x, "mxfp4"), wt)
    with pytest.raises(ValueError):
        w8.fp4_quantize(x[:, :40].contiguous())
    with pytest.raises(ValueError):
        w8.FP4Tensor(q.codes, q.scales[:, :, :256].contiguous(), q.factor, "nvfp4")
