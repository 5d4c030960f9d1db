"""The 4-bit linear layer and the norms around it: cases, plain forms and the framework's calls.

Operators
  quantize    BF16 rows to microscaled 4-bit floating point and back to the values the
              codes stand for (fp4_quantize, fp4_dequantize)
  linear      y = x W^T + bias with x quantised in the call and W held in 4 bits
              (fp4_linear)
  norm        the residual update between two blocks: the branch's RMSNorm, gate and
              residual scale, then the next block's RMSNorm with scale and shift
              (block_norm)
  norm_linear the same update with its output in 4 bits, multiplied by the next weight
              (block_norm_fp4, fp4_linear_prequant)

Formats: "mxfp4" has E2M1 elements in blocks of 32 along K with a power-of-two scale
(E8M0); "nvfp4" has E2M1 elements in blocks of 16 with an E4M3 scale, and one FP32 factor
a row.  Codes are packed two to a byte, the even element in the low half.  The block scales
lie in 512-byte tiles of 128 rows x 4 scales: tile [row / 128][block / 4], byte
16 (row % 32) + 4 (row % 128 / 32) + block % 4.
"""
import torch

own = False

EPS = 1e-6
SIZE = {"mxfp4": 32, "nvfp4": 16}      # elements a block
TINY = 2.0 ** -100                     # the least row maximum that nvfp4's row factor takes
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the activations of the MLP up-projection over a whole video's tokens
        dict(name="quantize nvfp4 16384x4096", op="quantize", format="nvfp4", M=16384, K=4096, x="student"),
        # the audio branch's tokens: rows that fill no 128-row tile
        dict(name="quantize mxfp4 1000x2048", op="quantize", format="mxfp4", M=1000, K=2048, x="normal"),
        # one token
        dict(name="quantize nvfp4 1x4096", op="quantize", format="nvfp4", M=1, K=4096, x="outliers"),
        # the MLP up-projection, the benchmark's own sizes
        dict(name="linear nvfp4 16384x4096x16384", op="linear", format="nvfp4", M=16384, K=4096, N=16384, x="student", bias=True),
        # an attention projection, with outlier channels
        dict(name="linear mxfp4 4096x4096x4096", op="linear", format="mxfp4", M=4096, K=4096, N=4096, x="outliers", bias=False),
        # ragged in every direction: M and N odd, K no multiple of 128
        dict(name="linear nvfp4 1000x2016x8191", op="linear", format="nvfp4", M=1000, K=2016, N=8191, x="normal", bias=True),
        # a few tokens: the weight's bytes count
        dict(name="linear mxfp4 37x2048x8192", op="linear", format="mxfp4", M=37, K=2048, N=8192, x="normal", bias=True),
        # one token
        dict(name="linear nvfp4 1x4096x16384", op="linear", format="nvfp4", M=1, K=4096, N=16384, x="outliers", bias=False),
        # the residual stream of the high-resolution chain, all factors, two samples
        dict(name="norm 32768x4096 modulated", op="norm", M=32768, K=4096, groups=2, post=True, modulated=True),
        # one token, norms and residual scale alone
        dict(name="norm 1x4096", op="norm", M=1, K=4096, groups=1, post=True, modulated=False),
        # a block's entry: the update, its 4-bit output and the QKV-sized product
        dict(name="norm_linear nvfp4 4096x4096", op="norm_linear", format="nvfp4", M=4096, K=4096, N=12288, groups=2, post=True, modulated=True),
        # the same on a handful of tokens, without the branch's norm
        dict(name="norm_linear mxfp4 6x2080", op="norm_linear", format="mxfp4", M=6, K=2080, N=4097, groups=3, post=False, modulated=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(("quantize", "linear", "linear", "norm", "norm_linear"))
    case = dict(op=op)
    if op != "norm":
        case["format"] = rng.choice(("mxfp4", "nvfp4"))
    M = _spread(rng, 1, 16384)
    K = 32 * _spread(rng, 1, 512)
    if op in ("quantize", "linear"):
        case["x"] = rng.choice(("normal", "student", "outliers"))
    if op in ("norm", "norm_linear"):
        case["groups"] = rng.choice([g for g in (1, 2, 3, 5, 8) if M % g == 0])
        case["post"], case["modulated"] = rng.random() < 0.7, rng.random() < 0.6
        if op == "norm":
            K = 8 * _spread(rng, 1, 2048)
    case["M"], case["K"] = M, K
    if op in ("linear", "norm_linear"):
        case["N"] = _spread(rng, 1, max(2, min(16384, 2 ** 40 // (M * K))))
    if op == "linear":
        case["bias"] = rng.random() < 0.5
    return case


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "quantize":      # x in, the values out
        return {"bytes": 4 * M * K, "flops": 4 * M * K}
    if case["op"] == "norm":          # h and the branch in, the new h and the norm out
        return {"bytes": 8 * M * K, "flops": 14 * M * K}
    N = case["N"]
    weight = N * K // 2 + N * K // SIZE[case["format"]] + 4 * N * (case["format"] == "nvfp4")
    if case["op"] == "linear":
        return {"bytes": 2 * M * K + weight + 2 * M * N + 2 * N * case["bias"], "flops": 2 * M * N * K}
    return {"bytes": 6 * M * K + weight + 2 * M * N, "flops": 2 * M * N * K + 14 * M * K}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _acts(kind, M, K, g):
    if kind == "student":             # heavy tails, three degrees of freedom
        z = torch.randn((4, M, K), generator=g, device="cuda")
        return (z[0] / (z[1:].square().sum(0) / 3).sqrt()).clamp(-64, 64).bfloat16()
    x = torch.randn((M, K), generator=g, device="cuda")
    if kind == "outliers":            # one channel in a hundred is 20 times the others
        x = x * torch.where(torch.rand((K,), generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.bfloat16()


def _normal(shape, g, scale=1.0, plus=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale + plus).bfloat16()


def prepare(case, seed):
    g = _gen(seed)
    M, K, op = case["M"], case["K"], case["op"]
    s = dict(case)
    if op in ("quantize", "linear"):
        s["x"] = _acts(case["x"], M, K, g)
    if op in ("linear", "norm_linear"):      # the weight as its file holds it
        N = case["N"]
        w = _normal((N, K), g, K ** -0.5)
        index, scales, factor = _quantize(w, case["format"])
        s["codes"] = _pack(index)
        s["scales"] = _tile(scales)
        s["factor"] = factor
        s["bias"] = _normal((N,), g, 0.01) if case.get("bias") else None
    if op in ("norm", "norm_linear"):
        B = case["groups"]
        s["h"] = _normal((M, K), g)
        s["y"] = _normal((M, K), g, 0.5)
        s["post_gamma"] = _normal((K,), g, 0.2, 1.0) if case["post"] else None
        s["pre_gamma"] = _normal((K,), g, 0.2, 1.0)
        mod = case["modulated"]
        s["gate"] = _normal((B, K), g, 0.5) if mod else None
        s["scale"] = _normal((B, K), g, 0.5) if mod else None
        s["shift"] = _normal((B, K), g, 0.5) if mod else None
        s["res_scale"] = 0.875
    return s


# ------------------------------------------------------------------ plain form
def _round_e2m1(a):
    """The index (0..7) of the level nearest to each a >= 0, ties to the even index."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0)).to(torch.uint8)


def _pow2(e):
    """2^e in 32 bits for whole numbers from -126 to 127, from the bits of a float."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantize(x, fmt):
    """Codes (4 bits, unpacked) [M, K], block scales as bytes [M, K / block], row factors."""
    M, K = x.shape
    B = SIZE[fmt]
    v = x.float().view(M, K // B, B)
    top = v.abs().amax(2)
    if fmt == "mxfp4":
        e = (torch.frexp(top)[1] - 3).clamp(-127, 127)        # floor(log2 top) - 2
        e = torch.where(top == 0, -127, e)
        index = _round_e2m1(v.abs() * _pow2(-e)[:, :, None])
        scales, factor = (e + 127).to(torch.uint8), None
    else:
        row = top.amax(1, keepdim=True).clamp(min=TINY)
        s = (top * 448 / row).to(torch.float8_e4m3fn)
        # a / (s * row / 2688), with both products exact in 32 bits
        q = (v.abs() * 0.65625) / (s.float() * (row / 4096))[:, :, None]
        index = torch.where(s.float()[:, :, None] == 0, 0, _round_e2m1(q))
        scales, factor = s.view(torch.uint8), (row / 2688).view(M)
    code = index + 8 * torch.signbit(v).to(torch.uint8)
    return code.view(M, K), scales, factor


def _pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _tile(s):
    """Block scales [rows, blocks] in tiles of 128 rows x 4, zeros past the end."""
    R, C = s.shape
    rt, ct = -(-R // 128), -(-C // 4)
    full = torch.zeros((rt * 128, ct * 4), dtype=torch.uint8, device=s.device)
    full[:R, :C] = s
    return full.view(rt, 4, 32, ct, 4).permute(0, 3, 2, 1, 4).reshape(rt, ct, 512).contiguous()


def _untile(t, R, C):
    rt, ct, _ = t.shape
    return t.view(rt, ct, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, ct * 4)[:R, :C]


def _values(code, scales, factor, fmt):
    """What codes (unpacked) stand for, in 32 bits."""
    M, K = code.shape
    table = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=code.device)
    v = table[code.int()].view(M, K // SIZE[fmt], SIZE[fmt])
    if fmt == "mxfp4":
        e = scales.int()[:, :, None] - 127
        v = v * 0.5 * _pow2((e + 1).clamp(max=127)) * torch.where(e == 127, 2.0, 1.0)
    else:
        v = v * scales.contiguous().view(torch.float8_e4m3fn).float()[:, :, None] * factor[:, None, None]
    return v.view(M, K)


def _weight_values(s):
    N, K = s["N"], s["K"]
    c = s["codes"]
    code = torch.stack((c & 15, c >> 4), 2).view(N, K)
    return _values(code, _untile(s["scales"], N, K // SIZE[s["format"]]), s["factor"], s["format"])


def _product(x, s):
    """x (values, 32 bits) times the weight, plus the bias, rounded once."""
    y = x @ _weight_values(s).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.bfloat16()


def _rstd(v):
    return (v.square().mean(1, keepdim=True) + EPS).rsqrt()


def _update(s):
    """(h', n): the residual after the branch, and the next block's normalised input."""
    M, K, B = s["M"], s["K"], s["groups"]
    rows = lambda t: t.float().repeat_interleave(M // B, 0)  # noqa: E731
    u = s["y"].float()
    if s["post_gamma"] is not None:
        u = u * _rstd(u) * s["post_gamma"].float()
    if s["gate"] is not None:
        u = rows(s["gate"]) * u
    h = (s["res_scale"] * s["h"].float() + u).bfloat16()
    n = h.float() * _rstd(h.float()) * s["pre_gamma"].float()
    if s["scale"] is not None:
        n = n * (1 + rows(s["scale"])) + rows(s["shift"])
    return h, n.bfloat16()


def run(s):
    op = s["op"]
    if own:
        import block_wise_w8a8_b200 as w8
        if op == "quantize":
            return w8.fp4_dequantize(w8.fp4_quantize(s["x"], s["format"]))
        norm = dict(post_gamma=s["post_gamma"], gate=s["gate"], pre_gamma=s["pre_gamma"], scale=s["scale"], shift=s["shift"],
                    res_scale=s["res_scale"], post_norm=s["post"], eps=EPS) if op in ("norm", "norm_linear") else None
        if op == "norm":
            return w8.block_norm(s["h"], s["y"], **norm)
        w = w8.FP4Weight(q=w8.FP4Tensor(s["codes"], s["scales"], s["factor"], s["format"]))
        if op == "linear":
            return w8.fp4_linear(s["x"], w, s["bias"])
        h, n = w8.block_norm_fp4(s["h"], s["y"], s["format"], **norm)
        return h, w8.fp4_linear_prequant(n, w, s["bias"])
    if op == "quantize":
        return _values(*_quantize(s["x"], s["format"]), s["format"]).bfloat16()
    if op == "norm":
        return _update(s)
    if op == "linear":
        return _product(_values(*_quantize(s["x"], s["format"]), s["format"]), s)
    h, n = _update(s)
    return h, _product(_values(*_quantize(n, s["format"]), s["format"]), s)


# ------------------------------------------------------------------ from the definition, in 64 bits
def _nearest(a):
    """The E2M1 value nearest to a (64 bits): steps of 0.5 up to 2, of 1 up to 4, of 2 above;
    torch.round takes ties to the even multiple, which is the even code."""
    a = a.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a)
    return (torch.round(a / step) * step).clamp(max=6)


def _exponent(a):
    """floor(log2 a) of normal 64-bit numbers a > 0, from their bits."""
    return ((a.view(torch.int64) >> 52) - 1023).double()


def _exact_values(x, fmt):
    """The values that x's codes stand for, from the formats' definition."""
    M, K = x.shape
    if fmt == "mxfp4":
        v = x.double().view(M, -1, 32)
        top = v.abs().amax(2, keepdim=True)
        e = _exponent(top) - 2
        e = torch.where(top > 0, e, -127.0).clamp(min=-127)
        out = torch.exp2(e) * _nearest(v * torch.exp2(-e))
    else:
        v = x.double().view(M, -1, 16)
        row = v.abs().amax((1, 2), keepdim=True).clamp(min=2.0 ** -100)
        t = v.abs().amax(2, keepdim=True) * 448 / row
        # E4M3: three bits after the leading one, steps of 2^-9 at least
        step = torch.exp2(_exponent(t.clamp(min=2.0 ** -6)) - 3)
        unit = torch.round(t / step) * step * row          # 2688 times the block's unit
        out = torch.where(unit > 0, unit / 2688 * _nearest(v * 2688 / unit), 0.0)
    return torch.copysign(out, v).view(M, K)


def _exact_weight(s):
    c, fmt, N, K = s["codes"].long(), s["format"], s["N"], s["K"]
    B = SIZE[fmt]
    level = torch.tensor(LEVELS, dtype=torch.float64, device=c.device)
    both = torch.stack((c % 16, c // 16), 2).view(N, K)
    v = level[both % 8] * (1 - 2 * (both // 8)).double()
    r = torch.arange(N, device=c.device)[:, None]
    b = torch.arange(K // B, device=c.device)[None, :]
    byte = s["scales"][r // 128, b // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4].double()
    if fmt == "mxfp4":
        scale = torch.exp2(byte - 127)
    else:
        e, m = byte // 8, byte % 8
        scale = torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), m * 2.0 ** -9) * s["factor"].double()[:, None]
    return v * scale.repeat_interleave(B, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_values(s["x"], s["format"])
    if op == "linear":
        y = _exact_values(s["x"], s["format"]) @ _exact_weight(s).T
        return y if s["bias"] is None else y + s["bias"].double()
    T = case["M"] // case["groups"]
    group = torch.arange(case["M"], device="cuda") // T
    u = s["y"].double()
    if s["post_gamma"] is not None:
        u = u / torch.sqrt((u * u).mean(1, keepdim=True) + EPS) * s["post_gamma"].double()
    if s["gate"] is not None:
        u = u * s["gate"].double()[group]
    h = s["h"].double() * s["res_scale"] + u
    kept = h.bfloat16().double()          # the residual is stored, and the next norm reads what is stored
    n = kept / torch.sqrt((kept * kept).mean(1, keepdim=True) + EPS) * s["pre_gamma"].double()
    if s["scale"] is not None:
        n = n * (1 + s["scale"].double()[group]) + s["shift"].double()[group]
    if op == "norm":
        return h, n
    return h, _exact_values(n.bfloat16(), s["format"]) @ _exact_weight(s).T
