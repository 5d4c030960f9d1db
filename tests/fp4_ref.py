"""Plain 64-bit reference of the microscaled 4-bit formats and of the fused block norm, on
torch tensors of any device.  Quotients are formed from products that are exact in 64 bits,
so each is rounded once, and a tie of the format is a tie here."""
import torch

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def exponent(a):
    """floor(log2 a) of positive normal doubles."""
    return ((a.contiguous().view(torch.int64) >> 52) & 2047) - 1023


def e2m1(a):
    """Index of the E2M1 level nearest |a|, ties to even, saturating."""
    a = a.abs()
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=a.device)
    up = torch.bucketize(a, edges, right=False)     # edges below a
    tie = torch.bucketize(a, edges, right=True)     # edges at or below a
    return torch.where((tie != up) & (up % 2 == 1), tie, up).to(torch.uint8)


def e4m3(a):
    """Byte of the E4M3 number nearest a >= 0 (ties to even, saturating at 448)."""
    e = exponent(a.clamp(min=2.0 ** -6))
    step = torch.exp2((e - 3).double())
    k = torch.round(a / step)                        # 8..16 of a normal, 0..8 of a subnormal
    v = (k * step).clamp(max=448.0)
    e = exponent(v.clamp(min=2.0 ** -6))
    k = v / torch.exp2((e - 3).double())
    return torch.where(k < 8, k, 8 * (e + 7).double() + k - 8).to(torch.uint8)


def e4m3_value(b):
    b = b.to(torch.int64)
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e > 0, torch.exp2((e - 7).double()) * (1 + m / 8), m * 2.0 ** -9)
    return torch.where((b & 127) == 127, torch.nan, v)


def quantize(x, fmt):
    """BF16 [M, K] -> codes (one a byte) [M, K], scale bytes [M, K / block], factor float32
    [M] or None."""
    M, K = x.shape
    B = BLOCK[fmt]
    v = x.double().view(M, K // B, B)
    ok = torch.isfinite(v)
    amax = torch.where(ok, v, 0.0).abs().amax(2)
    if fmt == "mxfp4":
        bad = ~ok.all(2)
        e = torch.where(amax > 0, exponent(torch.where(amax > 0, amax, 1.0)) - 2, -127).clamp(min=-127)
        code = e2m1(v * torch.exp2(-e.double())[:, :, None])
        scales = torch.where(bad, 255, e + 127).to(torch.uint8)
        dead, factor = bad[:, :, None], None
    else:
        bad = ~ok.view(M, -1).all(1)
        top = amax.amax(1).clamp(min=2.0 ** -100)
        scales = torch.where(bad[:, None], 0, e4m3(448 * amax / top[:, None]))
        unit = e4m3_value(scales) * top[:, None]
        code = torch.where(unit[:, :, None] > 0, e2m1(2688 * v / unit[:, :, None]), 0)
        factor = torch.where(bad, torch.nan, top / 2688).float()
        dead = bad[:, None, None]
    code = code.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return torch.where(dead, 0, code).view(M, K), scales, factor


def no_minus_zero(codes):
    """Packed codes with every -0 (8) as 0: nvfp4 leaves a zero's sign open."""
    low, high = codes & 15, codes >> 4
    return torch.where(low == 8, 0, low) | (torch.where(high == 8, 0, high) << 4)


def pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def unpack(codes):
    return torch.stack((codes & 15, codes >> 4), 2).view(codes.shape[0], -1)


def plain_scales(q):
    """The scale bytes [rows, blocks] of an FP4Tensor, by the layout's own formula."""
    nb = q.K // BLOCK[q.format]
    r = torch.arange(q.rows, device=q.codes.device)[:, None]
    b = torch.arange(nb, device=q.codes.device)[None, :]
    return q.scales[r // 128, b // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4]


def values(code, scales, factor, fmt, with_factor=True):
    """Doubles the codes stand for."""
    M, K = code.shape
    level = torch.tensor(LEVELS, dtype=torch.float64, device=code.device)
    v = level[(code & 7).long()] * (1 - 2 * (code >> 3).double())
    v = v.view(M, -1, BLOCK[fmt])
    if fmt == "mxfp4":
        s = torch.exp2(scales.double() - 127)
        s = torch.where(scales == 255, torch.nan, s)
    else:
        s = e4m3_value(scales)
        if with_factor:
            s = s * factor.double()[:, None]
    return (v * s[:, :, None]).view(M, K)


def tensor_values(q):
    return values(unpack(q.codes), plain_scales(q), q.factor, q.format)


def block_norm(h, y, post_gamma=None, gate=None, pre_gamma=None, scale=None, shift=None, *, res_scale=1.0,
               post_norm=True, eps=1e-6, h_kept=None):
    """(h', n) in 64 bits, unrounded; n from h' as stored (h_kept BF16, else h' rounded)."""
    M, K = h.shape
    rows = lambda t: t.double().repeat_interleave(M // t.shape[0], 0)  # noqa: E731
    rms = lambda v: (v * v).mean(1, keepdim=True).add(eps).sqrt()  # noqa: E731
    u = y.double()
    if post_norm:
        u = u / rms(u)
    if post_gamma is not None:
        u = u * post_gamma.double()
    if gate is not None:
        u = u * rows(gate)
    hh = h.double() * float(torch.tensor(res_scale)) + u
    kept = (hh.bfloat16() if h_kept is None else h_kept).double()
    n = kept / rms(kept)
    if pre_gamma is not None:
        n = n * pre_gamma.double()
    if scale is not None:
        n = n * (1 + rows(scale))
    if shift is not None:
        n = n + rows(shift)
    return hh, n
