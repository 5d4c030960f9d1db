"""The fused residual update and norms on the GPU against 64 bits, and the run of the
operators as a block uses them.

Tolerances: half a BF16 step of the result (2^-8 relative) for its one rounding, and FP32
arithmetic before it.  A row's squares are all positive, so their sum is off by at most
(adds in one chain) * 2^-24 of itself: K / 256 in a lane's own chain at the most, 10 more in
the tree; rstd takes half of that, and the products, the division and the root a few units
of 2^-24 each: together under (K / 256 + 40) * 2^-24 of the terms that are added up."""
import pytest
import torch

import block_wise_w8a8_b200 as w8
import fp4_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert w8.device_error() == 0


def _same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def _inputs(M, K, B, seed, post=True, gammas=True, mod=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    t = dict(h=r(M, K) * 3, y=r(M, K) * torch.exp(2 * r(M, 1)),
             post_gamma=1 + 0.3 * r(K) if post and gammas else None, pre_gamma=1 + 0.3 * r(K) if gammas else None,
             gate=r(B, K) if mod else None, scale=0.5 * r(B, K) if mod else None, shift=0.5 * r(B, K) if mod else None)
    return {k: None if v is None else v.bfloat16().cuda() for k, v in t.items()}


def _check(t, h2, n, K, res_scale=1.0, post_norm=True, eps=1e-6):
    hh, nn = ref.block_norm(**t, res_scale=res_scale, post_norm=post_norm, eps=eps, h_kept=h2)
    f32 = (K / 256 + 40) * 2.0 ** -24
    base = (t["h"].double() * res_scale).abs()
    tol = hh.abs() * 2.0 ** -8 + f32 * (base + (hh - t["h"].double() * res_scale).abs())
    assert bool(((h2.double() - hh).abs() <= tol).all()), float(((h2.double() - hh).abs() - tol).max())
    sh = 0 if t["shift"] is None else t["shift"].double().repeat_interleave(len(nn) // len(t["shift"]), 0)
    tol = nn.abs() * 2.0 ** -8 + f32 * ((nn - sh).abs() + (sh.abs() if t["shift"] is not None else 0))
    assert bool(((n.double() - nn).abs() <= tol).all()), float(((n.double() - nn).abs() - tol).max())


# many rows of each length that the ring takes, and the few-row form's lengths
SHAPES = [(9500, 24, 5), (9480, 512, 4), (4800, 1000, 3), (2400, 2048, 2), (1300, 4096, 1300), (1200, 2560, 1),
          (700, 8192, 7), (640, 10400, 2), (1, 8, 1), (3, 24, 3), (2, 32, 1), (17, 512, 1), (9, 520, 3), (10, 1024, 5), (12, 1000, 2), (300, 2048, 2),
          (7, 2080, 7), (130, 4096, 2), (5, 4104, 1), (6, 8192, 2), (3, 8200, 1), (4, 16384, 4), (2, 16392, 1),
          (3, 16416, 3), (2, 40000, 1), (2, 40008, 2)]


@pytest.mark.parametrize("M,K,B", SHAPES)
def test_all_factors(M, K, B):
    t = _inputs(M, K, B, M + K)
    h2, n = w8.block_norm(**t, res_scale=0.75, eps=1e-5)
    _check(t, h2, n, K, 0.75, True, 1e-5)
    # in place, with rows behind the last one left as they were
    big = torch.full((M + 1, K), 5.0, dtype=torch.bfloat16, device="cuda")
    big[:M] = t["h"]
    hv = big[:M]
    nb = torch.full((M + 1, K), 5.0, dtype=torch.bfloat16, device="cuda")
    out = w8.block_norm(**{**t, "h": hv}, res_scale=0.75, eps=1e-5, h_out=hv, n_out=nb[:M])
    assert out[0] is hv and _same(hv, h2) and _same(nb[:M], n)
    assert bool((big[M] == 5).all()) and bool((nb[M] == 5).all())


# rows whose length takes a number of warps that is no power of two
@pytest.mark.parametrize("M,K,B", [(3200, 1288, 4), (3300, 1536, 1), (2000, 2080, 5), (1900, 2560, 1900), (1600, 2880, 2),
                                   (1000, 4128, 8), (999, 5120, 1), (800, 6144, 4), (620, 12288, 5), (620, 12320, 4),
                                   (600, 16384, 600)])
def test_lengths_between_powers_of_two(M, K, B):
    t = _inputs(M, K, B, M + K)
    h2, n = w8.block_norm(**t, res_scale=0.75, eps=1e-5)
    _check(t, h2, n, K, 0.75, True, 1e-5)
    if K % 32:
        return
    for fmt in ("mxfp4", "nvfp4"):
        want = w8.fp4_quantize(n, fmt)
        h4, q = w8.block_norm_fp4(t["h"], t["y"], fmt, **{k: v for k, v in t.items() if k not in "hy"}, res_scale=0.75,
                                  eps=1e-5)
        assert _same(h4, h2)
        assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
        assert q.factor is None or torch.equal(q.factor, want.factor)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gammas", [True, False])
@pytest.mark.parametrize("mod", [True, False])
def test_left_out_factors(post, gammas, mod):
    for M, K in [(6, 768), (4, 4096), (2, 20000)]:
        t = _inputs(M, K, 2, K, post, gammas, mod)
        h2, n = w8.block_norm(**t, post_norm=post)
        _check(t, h2, n, K, post_norm=post)
    one = {**t, "gate": None, "shift": None}
    h2, n = w8.block_norm(**one, post_norm=post)
    _check(one, h2, n, K, post_norm=post)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,K,B", [s for s in SHAPES if s[1] % 32 == 0] + [(131, 96, 1), (9700, 320, 10),
                                                                          (4801, 992, 1)])
def test_fp4_output_is_the_two_calls(fmt, M, K, B):
    t = _inputs(M, K, B, M * 3 + K)
    h2, n = w8.block_norm(**t, res_scale=1.25)
    want = w8.fp4_quantize(n, fmt)
    h4, q = w8.block_norm_fp4(t.pop("h"), t.pop("y"), fmt, **t, res_scale=1.25)
    assert _same(h4, h2)
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
    assert q.factor is None or torch.equal(q.factor, want.factor)


def test_offsets_past_32_bits():
    M, K = 530000, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn((1000, K), generator=g, device="cuda").bfloat16().repeat(M // 1000, 1)
    y = h.flip(1)
    y[-5:] = torch.randn((5, K), generator=g, device="cuda").bfloat16()
    gamma = torch.randn((K,), generator=g, device="cuda").bfloat16()
    h2, n = w8.block_norm(h, y, post_gamma=gamma, pre_gamma=gamma)
    assert h.numel() > 2 ** 31
    for r in (0, 524287, 524288, M - 5, M - 1):
        t = dict(h=h[r:r + 1], y=y[r:r + 1], post_gamma=gamma, pre_gamma=gamma, gate=None, scale=None, shift=None)
        _check(t, h2[r:r + 1], n[r:r + 1], K)
    h4, q = w8.block_norm_fp4(h, y, "nvfp4", post_gamma=gamma, pre_gamma=gamma, h_out=h)
    assert _same(h4[-5:], h2[-5:])
    want = w8.fp4_quantize(n[-5:].contiguous())
    assert torch.equal(q.codes[-5:], want.codes)
    assert torch.equal(ref.plain_scales(q)[-5:], ref.plain_scales(want))


def test_zero_rows_and_infinities():
    t = _inputs(6, 256, 1, 4)
    t["y"][1] = 0
    t["h"][2] = 0
    t["y"][2] = 0
    t["y"][3, 7] = float("inf")
    t["h"][4, 9] = float("nan")
    h2, n = w8.block_norm(**t)
    hh, nn = ref.block_norm(**t, h_kept=h2)
    assert torch.equal(h2.isnan(), hh.isnan()) and torch.equal(n.isnan(), nn.isnan())
    ok = [0, 1, 2, 5]
    _check({k: v if v is None or k not in "hy" else v[ok] for k, v in t.items()}, h2[ok], n[ok], 256)
    _, q = w8.block_norm_fp4(t["h"], t["y"], "nvfp4", pre_gamma=t["pre_gamma"])
    assert bool(q.factor[3].isnan()) and bool(q.factor[4].isnan()) and bool(q.factor[ok].isfinite().all())
    z = torch.zeros((1, 64), dtype=torch.bfloat16, device="cuda")
    h2, n = w8.block_norm(z, z, eps=0.0)
    assert bool(h2.isnan().all()) and bool(n.isnan().all())
    h2, n = w8.block_norm(z, z, eps=1e-6)
    assert bool((h2 == 0).all()) and bool((n == 0).all())


def _block_run(M, T, fmt, seed):
    """Two blocks' worth: update and norm to 4 bits, product, update with its output."""
    K, N = 512, 1024
    t = _inputs(M, K, M // T, seed)
    g = torch.Generator().manual_seed(seed)
    up = w8.FP4Weight((torch.randn((N, K), generator=g) * K ** -0.5).bfloat16().cuda(), fmt)
    down = w8.FP4Weight((torch.randn((K, N), generator=g) * N ** -0.5).bfloat16().cuda(), fmt)
    args = {k: v for k, v in t.items() if k not in "hy"}

    def run(h, y):
        h, q = w8.block_norm_fp4(h, y, fmt, **args)
        u = w8.fp4_linear_prequant(q, up)
        y = w8.fp4_linear(u, down)
        return w8.block_norm(h, y, **args)
    return t, args, up, down, run


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,T", [(1, 1), (6, 3), (260, 130)])
def test_operators_in_a_row(fmt, M, T):
    """The chain against the 64-bit formulas on the values that each step's input holds.
    A step rounds to BF16 (2^-8) what a 64-bit chain with the same 4-bit codes computes; its
    product's tolerance is that of the linear's own tests."""
    t, args, up, down, run = _block_run(M, T, fmt, M + 1)
    h3, n3 = run(t["h"], t["y"])
    h2, q = w8.block_norm_fp4(t["h"], t["y"], fmt, **args)
    _, n = w8.block_norm(t["h"], t["y"], **args)
    _check(t, h2, n, 512)
    code, scales, factor = ref.quantize(n.cpu(), fmt)
    assert torch.equal(ref.no_minus_zero(q.codes.cpu()), ref.no_minus_zero(ref.pack(code)))
    assert torch.equal(ref.plain_scales(q).cpu(), scales)
    y = n.double()
    for qx, wt, K in ((q, up, 512), (None, down, 1024)):
        if qx is None:
            qx = w8.fp4_quantize(u, fmt)  # noqa: F821
        xv, wv = ref.tensor_values(qx), ref.tensor_values(wt.q)
        want, size = xv @ wv.T, xv.abs() @ wv.abs().T
        u = w8.fp4_linear_prequant(qx, wt)
        assert bool(((u.double() - want).abs() <= want.abs() * 2.0 ** -8 + size * (K / 64 + 8) * 2.0 ** -22).all())
    _check({**t, "h": h2, "y": u}, h3, n3, 512)
    assert y.shape == (M, 512)


def test_chain_captured_and_replayed():
    t, args, up, down, run = _block_run(48, 24, "nvfp4", 9)
    want = run(t["h"], t["y"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(t["h"], t["y"])
    graph.replay()
    assert _same(out[0], want[0]) and _same(out[1], want[1])
    t["y"].copy_(t["y"].flip(0))
    graph.replay()
    want = run(t["h"], t["y"])
    assert _same(out[0], want[0]) and _same(out[1], want[1])


def test_refusals():
    t = _inputs(4, 64, 2, 1)
    with pytest.raises(ValueError):
        w8.block_norm(**t, post_norm=False)                              # post_gamma without post_norm
    with pytest.raises(ValueError):
        w8.block_norm(**{**t, "scale": t["scale"][:1]})                  # gate has two rows
    with pytest.raises(ValueError):
        w8.block_norm(**{**t, "gate": None, "scale": None, "shift": t["h"][:3]})      # 3 does not divide 4
    with pytest.raises(ValueError):
        w8.block_norm(t["h"], t["y"][:2])
    with pytest.raises(ValueError):
        w8.block_norm(t["h"].t(), t["y"].t())
    with pytest.raises(TypeError):
        w8.block_norm(t["h"].float(), t["y"].float())
    with pytest.raises(ValueError):
        w8.block_norm_fp4(t["h"][:, :40].contiguous(), t["y"][:, :40].contiguous())
    with pytest.raises(w8.W8A8Error) as e:
        w8.block_norm(t["h"][:, :4].contiguous(), t["y"][:, :4].contiguous())
    assert e.value.code == 2
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(res_scale=float("inf"))):
        with pytest.raises(w8.W8A8Error) as e:
            w8.block_norm(t["h"], t["y"], **bad)
        assert e.value.code == 1
    empty = t["h"][:0]
    h2, n = w8.block_norm(empty, empty)
    assert h2.shape == n.shape == (0, 64)
    h2, q = w8.block_norm_fp4(empty, empty)
    assert q.codes.shape == (0, 32)
