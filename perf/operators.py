"""Cases for timing and checking the 8-bit activation operators.

Five operators that belong together: the input of a linear layer is kept in
8 bits for the backward pass, and the same 8-bit copy is the left operand of
an 8-bit frozen weight's product.

  quant       8-bit block codes of a bf16 matrix, and their decoding
  swiglu      the MLP's activation with its checkpoints in 8 bits: forward
              (h, and the codes of h, g and u) and backward (from the codes)
  nf4_bwd     backward of the NF4 linear layer from an 8-bit input
  fp8_fwd     product of 8-bit blocks (scale per 128), with the adapter term
  fp8_bwd     its backward pass

The 8-bit format (both operands): a row of K values is cut into blocks of 128
(the tail is padded with zeros), each block has one scale 2^e, kept as the
byte e + 127, and a value x is held as the nearest E4M3 (or E5M2) code of
x / 2^e, ties to even, where e is the least exponent >= -110 with
max|x| <= 448 * 2^e (57344 * 2^e for E5M2; the maximum is over the block's
finite values). A weight has one scale for each 128 x 128 block, and is also
kept transposed. Row stride of the codes: K rounded up to 128; of the scales:
K / 128 rounded up to a multiple of 4.
"""

import math

import torch

own = False

BLOCK = 128
E4M3, E5M2 = 0, 1
# format -> (exponent bias, mantissa bits, largest binary exponent, largest value / 2^that)
FORMATS = {E4M3: (7, 3, 8, 1.75), E5M2: (15, 2, 15, 1.75)}
E_MIN = -110

# 16 NF4 levels (normal quantiles of equal mass per half, endpoints -1 and 1)
NF4 = [float.fromhex(v) for v in (
    "-0x1.0p+0 -0x1.647362p-1 -0x1.0cd65cp-1 -0x1.94653cp-2 -0x1.234496p-2 -0x1.7a6a7ap-3 "
    "-0x1.74f0d2p-4 0x0.0p+0 0x1.45f602p-4 0x1.4995bep-3 0x1.f809b4p-3 0x1.5a066cp-2 "
    "0x1.c3496ap-2 0x1.200f52p-1 0x1.722760p-1 0x1.0p+0").split()]


def up(a, b):
    return (a + b - 1) // b * b


def code_values(fmt):
    """The value of each of the 256 codes, from the format's bit layout."""
    bias, mb, _, _ = FORMATS[fmt]
    eb = 7 - mb
    out = []
    for c in range(256):
        s, ex, man = c >> 7, (c >> mb) & ((1 << eb) - 1), c & ((1 << mb) - 1)
        if fmt == E4M3 and (c & 127) == 127:
            v = math.nan
        elif fmt == E5M2 and ex == 31:
            v = math.inf if man == 0 else math.nan
        elif ex == 0:
            v = man * 2.0 ** (1 - bias - mb)
        else:
            v = (1 + man / (1 << mb)) * 2.0 ** (ex - bias)
        out.append(-v if s else v)
    return out


# ---------------------------------------------------------------------------
# the cases

def listed():
    return [
        # a decode batch: 16 tokens of a 4096-wide model, where a call's latency counts
        dict(name="quant-16x4096", op="quant", M=16, K=4096, fmt=E4M3),
        # the down projection's input of a 7B-shaped MLP at 2048 tokens
        dict(name="quant-2048x11008", op="quant", M=2048, K=11008, fmt=E4M3),
        # a short ragged prompt; gate and up side by side in one buffer
        dict(name="swiglu-fwd-17x11008", op="swiglu_fwd", M=17, F=11008, joined=True, fmt=E4M3),
        # the 7B-shaped MLP's activation in a training step, both directions
        dict(name="swiglu-fwd-2048x11008", op="swiglu_fwd", M=2048, F=11008, joined=False, fmt=E4M3),
        dict(name="swiglu-bwd-2048x11008", op="swiglu_bwd", M=2048, F=11008, joined=False, fmt=E4M3),
        # the smallest layer: 16 tokens through 256 x 256 with a rank-8 adapter
        dict(name="nf4-bwd-16x256x256", op="nf4_bwd", M=16, N=256, K=256, r=8, drop=0.0,
             fmt=E4M3),
        # the gate projection's backward at 2048 tokens under LoRA dropout
        dict(name="nf4-bwd-2048x11008x4096", op="nf4_bwd", M=2048, N=11008, K=4096, r=64,
             drop=0.05, fmt=E4M3),
        # one token through a 4096 x 4096 projection
        dict(name="fp8-fwd-1x4096x4096", op="fp8_fwd", M=1, N=4096, K=4096, r=16, fmt=E4M3),
        # odd sizes on every side, no adapter, E5M2 activations
        dict(name="fp8-fwd-333x1001x1544", op="fp8_fwd", M=333, N=1001, K=1544, r=0, fmt=E5M2),
        # 65B-shaped up projection at 4096 tokens: the largest product
        dict(name="fp8-fwd-4096x22016x8192", op="fp8_fwd", M=4096, N=22016, K=8192, r=64,
             fmt=E4M3),
        # a short batch through an attention projection, both gradients
        dict(name="fp8-bwd-257x4096x4096", op="fp8_bwd", M=257, N=4096, K=4096, r=8, fmt=E5M2),
        # the down projection's backward at 2048 tokens
        dict(name="fp8-bwd-2048x4096x11008", op="fp8_bwd", M=2048, N=4096, K=11008, r=64,
             fmt=E4M3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "swiglu_fwd", "swiglu_bwd", "nf4_bwd", "fp8_fwd", "fp8_fwd",
                     "fp8_bwd"])
    fmt = rng.choice([E4M3, E5M2])
    if op == "quant":
        return dict(op=op, M=_log(rng, 1, 4096), K=_log(rng, 64, 22016), fmt=fmt)
    if op.startswith("swiglu"):
        return dict(op=op, M=_log(rng, 1, 4096), F=_log(rng, 64, 22016),
                    joined=rng.random() < 0.5, fmt=fmt)
    M = _log(rng, 1, 4096)
    r = rng.choice([1, 4, 8, 16, 24, 32, 64, 100, 128])
    N, K = 64 * _log(rng, 1, 200), 64 * _log(rng, 1, 150)
    if op == "nf4_bwd":
        return dict(op=op, M=M, N=N, K=K, r=r, drop=rng.choice([0.0, 0.05, 0.1]), fmt=fmt)
    if op == "fp8_fwd" and rng.random() < 0.4:  # the plain product takes any size
        return dict(op=op, M=M, N=_log(rng, 1, 12000), K=_log(rng, 1, 9000), r=0, fmt=fmt)
    return dict(op=op, M=M, N=N, K=K, r=r, fmt=fmt)


def work(case):
    op = case["op"]
    if op == "quant":  # read bf16; write codes and scales; read them; write bf16
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (2 + 1 + 1 + 2) + 2 * M * K / BLOCK, "flops": 4.0 * M * K}
    if op == "swiglu_fwd":  # read g, u; write h and three 8-bit copies; decode the three
        M, F = case["M"], case["F"]
        return {"bytes": M * F * (4 + 2 + 3 + 3 + 6), "flops": 20.0 * M * F}
    if op == "swiglu_bwd":
        M, F = case["M"], case["F"]
        return {"bytes": M * F * (2 + 2 + 4), "flops": 20.0 * M * F}
    M, N, K, r = (case[k] for k in ("M", "N", "K", "r"))
    if op == "nf4_bwd":
        return {"bytes": 2 * M * N + M * K + N * K / 2 + N * K / 64 + 2 * M * K
                + 6 * r * (N + K) + 4 * M * r + (M * K / 8 if case["drop"] else 0),
                "flops": 2.0 * M * N * K + 2.0 * M * r * (2 * N + 2 * K)}
    if op == "fp8_fwd":
        return {"bytes": M * K + N * K + 2 * M * N + 2 * r * (N + K) + 4 * M * r,
                "flops": 2.0 * M * N * K + 2.0 * M * r * (N + K)}
    return {"bytes": 2 * M * N + M * K + N * K + 2 * M * K + 6 * r * (N + K) + 4 * M * r,
            "flops": 2.0 * M * N * K + 2.0 * M * r * (2 * N + 2 * K)}


# ---------------------------------------------------------------------------
# inputs

class Draw:
    """Seeded tensors on the GPU."""

    def __init__(self, seed):
        self.dev = torch.device("cuda", torch.cuda.current_device())
        self.g = torch.Generator(device=self.dev)
        self.g.manual_seed(seed)

    def normal(self, shape, std):
        return torch.randn(shape, generator=self.g, device=self.dev) * std

    def activation(self, M, K):
        """N(0, 1) with a few columns far larger, as a decoder's activations have."""
        x = self.normal((M, K), 1.0)
        wide = torch.rand(K, generator=self.g, device=self.dev) < 0.005
        return (x * torch.where(wide, 20.0, 1.0)).to(torch.bfloat16)

    def integers(self, lo, hi, shape, dtype=torch.uint8):
        return torch.randint(lo, hi, shape, generator=self.g, device=self.dev, dtype=dtype)


def encode(x, fmt, rows):
    """8-bit codes and scale bytes of x [R x C]; one scale per `rows` x 128 block."""
    R, C = x.shape
    Rp, Cp = up(R, rows), up(C, BLOCK)
    p = torch.zeros(Rp, Cp, dtype=torch.float32, device=x.device)
    p[:R, :C] = x
    blk = p.view(Rp // rows, rows, Cp // BLOCK, BLOCK)
    _, _, top, frac = FORMATS[fmt]
    m, ex = torch.frexp(blk.abs().amax(dim=(1, 3)))
    e = ex - 1 - top + (2 * m > frac).int()
    e = torch.where(m == 0, torch.full_like(e, E_MIN), e).clamp(min=E_MIN)
    y = (blk.double() * torch.pow(2.0, -e.double())[:, None, :, None]).float()
    dt = torch.float8_e4m3fn if fmt == E4M3 else torch.float8_e5m2
    codes = y.to(dt).view(torch.uint8).view(Rp, Cp)[:R].contiguous()
    scales = torch.zeros(Rp // rows, up(Cp // BLOCK, 4), dtype=torch.uint8, device=x.device)
    scales[:, :Cp // BLOCK] = (e + 127).to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    d = Draw(seed)
    op, fmt = case["op"], case["fmt"]
    s = dict(case)
    # decoding tables: 256 code values, 256 scales, 2^i for i in [-200, 200]
    s["lut"] = torch.tensor(code_values(fmt), dtype=torch.float32, device=d.dev)
    s["lut_w"] = torch.tensor(code_values(E4M3), dtype=torch.float32, device=d.dev)
    s["lut_s"] = torch.tensor([2.0 ** (i - 127) for i in range(255)] + [math.nan],
                              dtype=torch.float32, device=d.dev)
    s["pow2"] = torch.tensor([2.0 ** max(-149, min(127, i)) for i in range(-200, 201)],
                             dtype=torch.float32, device=d.dev)
    if op == "quant":
        s["x"] = d.activation(case["M"], case["K"])
        return s
    if op.startswith("swiglu"):
        M, F = case["M"], case["F"]
        gu = torch.empty(M, 2 * F, dtype=torch.bfloat16, device=d.dev)
        gu[:, :F] = d.normal((M, F), 1.5)
        gu[:, F:] = d.normal((M, F), 1.0)
        if op == "swiglu_fwd":
            s["g"], s["u"] = gu[:, :F], gu[:, F:]
            if not case["joined"]:
                s["g"], s["u"] = s["g"].contiguous(), s["u"].contiguous()
            return s
        s["g8"], s["gs"] = encode(gu[:, :F], fmt, 1)
        s["u8"], s["us"] = encode(gu[:, F:], fmt, 1)
        s["dh"] = d.normal((M, F), 1e-3).to(torch.bfloat16)
        # where joined, the two gradients are the halves of one buffer
        both = torch.empty(M, 2 * F, dtype=torch.bfloat16, device=d.dev)
        s["dg"], s["du"] = (both[:, :F], both[:, F:]) if case["joined"] else (
            torch.empty(M, F, dtype=torch.bfloat16, device=d.dev),
            torch.empty(M, F, dtype=torch.bfloat16, device=d.dev))
        return s
    M, N, K, r = (case[k] for k in ("M", "N", "K", "r"))
    x = d.activation(M, K)
    s["x8"], s["xs"] = encode(x, fmt, 1)
    s["scale"] = 2.0
    s["A"] = d.normal((K, r), 0.01).to(torch.bfloat16) if r else None
    s["B"] = d.normal((r, N), 0.01).to(torch.bfloat16) if r else None
    if op == "nf4_bwd":
        n = N * K
        s["codes"] = d.integers(0, 256, (n // 2,))
        s["absmax_q"] = d.integers(120, 256, (n // 64,))
        s["absmax_s2"] = torch.rand((n // 64 + 255) // 256, generator=d.g, device=d.dev) * 0.02 + 0.07
        s["nf4"] = torch.tensor(NF4, dtype=torch.float32, device=d.dev)
        if case["drop"]:
            keep = torch.rand(M, K, generator=d.g, device=d.dev) >= case["drop"]
            w = torch.tensor([1 << i for i in range(32)], dtype=torch.int64, device=d.dev)
            bits = (keep.view(M, K // 32, 32) * w).sum(-1)
            s["keep"] = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32)
    else:
        w = d.normal((N, K), 0.02)
        s["w8"], s["ws"] = encode(w, E4M3, BLOCK)
        s["w8t"], s["wst"] = encode(w.t().contiguous(), E4M3, BLOCK) if op == "fp8_bwd" else (None, None)
    if op != "fp8_fwd":
        s["dY"] = d.normal((M, N), 1e-3).to(torch.bfloat16)
        # T is what the forward kept: (kept X) A in float32
        X = rows_f32(s["x8"], s["xs"], K, s)
        s["T"] = masked(X, s) @ s["A"].float()
    return s


# ---------------------------------------------------------------------------
# the plain form

def rows_f32(codes, scales, C, s, lut="lut"):
    """float32 values of an 8-bit matrix with one scale per row and 128 columns."""
    R, Cp = codes.shape
    v = s[lut][codes.int()].view(R, Cp // BLOCK, BLOCK)
    return (v * s["lut_s"][scales[:, :Cp // BLOCK].int()][:, :, None]).view(R, Cp)[:, :C]


def weight_f32(s, N, K):
    codes, scales = s["w8"], s["ws"]
    rows = scales[torch.arange(N, device=codes.device) // BLOCK]
    return rows_f32(codes, rows, K, s, "lut_w")


def masked(X, s):
    """D(X): the kept elements times the inverse keep probability."""
    if not s.get("drop"):
        return X
    thr = math.floor(s["drop"] * 65536 + 0.5)
    bit = torch.arange(32, device=X.device, dtype=torch.int32)
    keep = ((s["keep"][:, :, None] >> bit) & 1).view(X.shape)
    return X * keep * (65536.0 / (65536 - thr))


def round_blocks(x, s, fmt):
    """The values that the 8-bit codes of x [R x C] stand for (float32 in and out)."""
    R, C = x.shape
    Cp = up(C, BLOCK)
    bias, mb, top, frac = FORMATS[fmt]
    p = torch.zeros(R, Cp, dtype=torch.float32, device=x.device)
    p[:, :C] = x
    p = p.view(R, Cp // BLOCK, BLOCK)
    m, ex = torch.frexp(p.abs().amax(dim=2, keepdim=True))
    e = ex - 1 - top + (2 * m > frac).int()
    e = torch.where(m == 0, torch.full_like(e, E_MIN), e).clamp(min=E_MIN)
    y = p * s["pow2"][(200 - e).long()]
    _, ey = torch.frexp(y)
    step = (ey - 1).clamp(min=1 - bias) - mb  # exponent of the spacing at y
    q = torch.round(y * s["pow2"][(200 - step).long()]) * s["pow2"][(200 + step).long()]
    return (q * s["pow2"][(200 + e).long()]).view(R, Cp)[:, :C]


def sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def nf4_f32(s, N, K):
    """bf16-rounded dequantized NF4 weight, in float32."""
    c = s["codes"].int()
    lv = torch.stack([s["nf4"][c & 15], s["nf4"][c >> 4]], dim=1).view(-1, 64)
    b = torch.arange(N * K // 64, device=c.device)
    cst = s["absmax_q"].float() / 255.0 * s["absmax_s2"][b // 256]
    return (lv * cst[:, None]).to(torch.bfloat16).float().view(N, K)


def adapter_grads(s, X, dY):
    """(G = dY B^T, dA, dB) in float32."""
    D = masked(X, s)
    G = dY @ s["B"].float().t()
    return G, s["scale"] * (D.t() @ G), s["scale"] * (s["T"].t() @ dY)


def plain(s):
    op, fmt = s["op"], s["fmt"]
    bf = torch.bfloat16
    if op == "quant":
        return {"x": round_blocks(s["x"].float(), s, fmt).to(bf)}
    if op == "swiglu_fwd":
        g, u = s["g"].float(), s["u"].float()
        h = (g * sigmoid(g) * u).to(bf)
        return {"h": h, "h8": round_blocks(h.float(), s, fmt).to(bf),
                "g8": round_blocks(g, s, fmt).to(bf), "u8": round_blocks(u, s, fmt).to(bf)}
    if op == "swiglu_bwd":
        F = s["F"]
        g, u = rows_f32(s["g8"], s["gs"], F, s), rows_f32(s["u8"], s["us"], F, s)
        dh, p = s["dh"].float(), sigmoid(g)
        return {"dg": (dh * u * (p * (1.0 + g * (1.0 - p)))).to(bf), "du": (dh * (g * p)).to(bf)}
    N, K, r = s["N"], s["K"], s["r"]
    X = rows_f32(s["x8"], s["xs"], K, s)
    if op == "fp8_fwd":
        Y = X @ weight_f32(s, N, K).t()
        if not r:
            return {"Y": Y.to(bf)}
        T = X @ s["A"].float()
        return {"Y": (Y + s["scale"] * (T @ s["B"].float())).to(bf), "T": T}
    dY = s["dY"].float()
    G, dA, dB = adapter_grads(s, X, dY)
    low = s["scale"] * (G @ s["A"].float().t())
    if op == "nf4_bwd":
        return {"dX": (dY @ nf4_f32(s, N, K) + masked(low, s)).to(bf), "dA": dA, "dB": dB}
    dX = round_blocks(dY, s, fmt) @ weight_f32(s, N, K) + low
    return {"dX": dX.to(bf), "dA": dA, "dB": dB}


# ---------------------------------------------------------------------------
# the framework's calls

def run(s):
    if not own:
        return plain(s)
    import bit_quantized_finetuning_quantize_amd as q
    op, fmt = s["op"], s["fmt"]
    if op == "quant":
        return {"x": q.qlora_act8_dequantize(q.qlora_act8_quantize(s["x"], fmt))}
    if op == "swiglu_fwd":
        h, h8, g8, u8 = q.qlora_swiglu_act8_fwd(s["g"], s["u"], fmt)
        dec = q.qlora_act8_dequantize
        return {"h": h, "h8": dec(h8), "g8": dec(g8), "u8": dec(u8)}
    if op == "swiglu_bwd":
        shape = (s["M"], s["F"])
        dg, du = q.qlora_swiglu_act8_bwd(s["dh"], q.Act8(s["g8"], s["gs"], shape, fmt),
                                         q.Act8(s["u8"], s["us"], shape, fmt), s["dg"], s["du"])
        return {"dg": dg, "du": du}
    M, N, K, r = s["M"], s["N"], s["K"], s["r"]
    x8 = q.Act8(s["x8"], s["xs"], (M, K), fmt)
    if "wsp" not in s:  # the workspace that a training or serving loop keeps
        s["wsp"] = q.act8_workspace(M, N, K, r, s["x8"].device)
    if op == "nf4_bwd":
        w = q.Nf4Store(s["codes"], s["absmax_q"], s["absmax_s2"], N * K, (N, K))
        dX, dA, dB = q.qlora_linear_bwd_act8(s["dY"], x8, s["T"], w, s["A"], s["B"], s["scale"],
                                             keep_mask=s.get("keep"), p=s["drop"], ws=s["wsp"])
        return {"dX": dX, "dA": dA, "dB": dB}
    w = q.Fp8Weight(s["w8"], s["ws"], s["w8t"], s["wst"], (N, K))
    if op == "fp8_fwd":
        Y, T = q.qlora_fp8_linear_fwd(x8, w, s["A"], s["B"], s["scale"], ws=s["wsp"])
        return {"Y": Y, "T": T} if r else {"Y": Y}
    dX, dA, dB = q.qlora_fp8_linear_bwd(s["dY"], x8, s["T"], w, s["A"], s["B"], s["scale"], fmt,
                                        ws=s["wsp"])
    return {"dX": dX, "dA": dA, "dB": dB}


# ---------------------------------------------------------------------------
# the definition in 64 bits, apart from the plain form: values are looked up
# by distance among all codes, matrices are decoded block by block, and the
# sums are float64 products

def _nearest(x, fmt):
    """What the codes of x [R x C] (float64) stand for."""
    R, C = x.shape
    vals = sorted(v for v in code_values(fmt)[:128] if math.isfinite(v))
    grid = torch.tensor(vals, dtype=torch.float64, device=x.device)
    mids = (grid[1:] + grid[:-1]) / 2
    out = torch.empty_like(x)
    exps = torch.arange(E_MIN, 128, device=x.device, dtype=torch.float64)
    limits = vals[-1] * torch.exp2(exps)
    for c in range(0, C, BLOCK):
        b = x[:, c:c + BLOCK]
        # least exponent whose largest value covers the block
        at = torch.searchsorted(limits, b.abs().amax(dim=1)).clamp(max=exps.numel() - 1)
        unit = torch.exp2(exps[at])[:, None]
        y = b.abs() / unit
        lo = torch.searchsorted(mids, y)  # a tie stays at the lower code
        hi = torch.searchsorted(mids, y, right=True)
        code = torch.where(lo % 2 == 0, lo, hi)  # of a tie's two codes, the even one
        out[:, c:c + BLOCK] = torch.copysign(grid[code], b) * unit
    return out


def _decode(codes, scales, fmt, C, rows):
    """float64 values of codes with one scale per `rows` x 128 block."""
    v = torch.tensor(code_values(fmt), dtype=torch.float64, device=codes.device)
    x = torch.empty(codes.shape[0], C, dtype=torch.float64, device=codes.device)
    unit = torch.exp2(scales.double() - 127).repeat_interleave(rows, 0)[:codes.shape[0]]
    for c in range(0, C, BLOCK):
        x[:, c:c + BLOCK] = v[codes[:, c:min(c + BLOCK, C)].long()] * unit[:, c // BLOCK, None]
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt = s["op"], s["fmt"]
    if op == "quant":
        return {"x": _nearest(s["x"].double(), fmt)}
    if op == "swiglu_fwd":
        g, u = s["g"].double(), s["u"].double()
        h = g * torch.special.expit(g) * u
        return {"h": h, "h8": _nearest(h.to(torch.bfloat16).double(), fmt),
                "g8": _nearest(g, fmt), "u8": _nearest(u, fmt)}
    if op == "swiglu_bwd":
        g = _decode(s["g8"], s["gs"], fmt, s["F"], 1)
        u = _decode(s["u8"], s["us"], fmt, s["F"], 1)
        p = torch.special.expit(g)
        dh = s["dh"].double()
        return {"dg": dh * u * p * (1 + g * torch.special.expit(-g)), "du": dh * g * p}
    N, K, r = s["N"], s["K"], s["r"]
    X = _decode(s["x8"], s["xs"], fmt, K, 1)
    A = s["A"].double() if r else None
    B = s["B"].double() if r else None
    if op == "fp8_fwd":
        Y = X @ _decode(s["w8"], s["ws"], E4M3, K, BLOCK).T.contiguous()
        if not r:
            return {"Y": Y}
        T = X @ A
        return {"Y": Y + s["scale"] * (T @ B), "T": T}
    dY = s["dY"].double()
    D = X
    keep = 1.0
    if s.get("drop"):
        word = s["keep"].long() & 0xffffffff
        keep = torch.stack([(word >> i) & 1 for i in range(32)], dim=2).view(X.shape).double()
        keep = keep / (1 - math.floor(s["drop"] * 65536 + 0.5) / 65536)
        D = X * keep
    G = dY @ B.T.contiguous()
    low = s["scale"] * (G @ A.T.contiguous()) * keep
    dA = s["scale"] * (D.T.contiguous() @ G)
    dB = s["scale"] * (s["T"].double().T.contiguous() @ dY)
    if op == "nf4_bwd":
        lv = torch.tensor(NF4, dtype=torch.float32, device=X.device)
        lo, hi = s["codes"].long() % 16, s["codes"].long() // 16
        level = torch.empty(N * K, dtype=torch.float32, device=X.device)
        level[0::2], level[1::2] = lv[lo], lv[hi]
        # the stored weight: two float32 products, then one rounding to bf16
        c = (s["absmax_q"].float() / 255) * s["absmax_s2"].repeat_interleave(256)[:N * K // 64]
        W = (level * c.repeat_interleave(64)).to(torch.bfloat16).double().view(N, K)
        return {"dX": dY @ W + low, "dA": dA, "dB": dB}
    W = _decode(s["w8"], s["ws"], E4M3, K, BLOCK)
    return {"dX": _nearest(dY, fmt) @ W + low, "dA": dA, "dB": dB}
