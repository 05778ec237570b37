"""What is timed of the microscaled 4-bit operators: the cases, their inputs and the operators' plain forms.

MXFP4: elements of E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), one E8M0 scale (a power of two) for each 32
elements of a row.  NVFP4: the same elements, one E4M3 scale for each 16 and one float per tensor.  Two elements lie in a
byte, the even one in the low nibble.  Scale bytes lie in tiles of 128 rows by 4 scales: byte (r % 32) * 16 + (r / 32) * 4 + c
of a tile of 512 bytes, tiles row-major.  The rows of an expert begin a tile of their own: tile row
offsets[e] / 128 + e + (row - offsets[e]) / 128.

Kinds of cases:
  quantize   a matrix to MXFP4 and back to the values that the codes stand for
  linear     activations quantized to MXFP4 and multiplied with MXFP4 weights, in one call
  nvfp4      packed NVFP4 activations (row-major scales, as the quantizers write them) times NVFP4 weights
  experts    rows sorted by expert, quantized to MXFP4 and multiplied with their expert's MXFP4 weights
"gate": the weights' rows alternate gate and up, and silu(gate) * up is written.
"""
import math
import random

import torch

own = False

F32, F64 = torch.float32, torch.float64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the activations of a batch of 16 tokens before a 4096-wide layer: one small call
        dict(name="quantize 16x4096", kind="quantize", M=16, K=4096, dtype="bf16", out="bf16"),
        # the activations of a prompt, with outlier channels
        dict(name="quantize 2048x4096", kind="quantize", M=2048, K=4096, dtype="bf16", out="bf16"),
        # a weight matrix, once when a model is packed
        dict(name="quantize 14336x4096", kind="quantize", M=14336, K=4096, dtype="f16", out="f32"),
        # one token through a square projection: latency and the weights' bytes
        dict(name="linear 1x4096x4096", kind="linear", M=1, N=4096, K=4096, dtype="bf16", out="bf16", gate=False),
        # a batch of tokens through the widening projection
        dict(name="linear 16x14336x4096", kind="linear", M=16, N=14336, K=4096, dtype="f16", out="f16", gate=False),
        # sizes that no tile divides
        dict(name="linear 333x1000x2080", kind="linear", M=333, N=1000, K=2080, dtype="bf16", out="bf16", gate=False),
        # a chunk of a prompt through a gated pair of projections
        dict(name="gated 512x28672x4096", kind="linear", M=512, N=28672, K=4096, dtype="bf16", out="bf16", gate=True),
        # a long prompt through the widening projection
        dict(name="linear 4096x14336x4096", kind="linear", M=4096, N=14336, K=4096, dtype="bf16", out="bf16", gate=False),
        # a few tokens through a large model's projection, packed NVFP4
        dict(name="nvfp4 4x28672x8192", kind="nvfp4", M=4, N=28672, K=8192, out="f16"),
        # a prompt through the narrowing projection, packed NVFP4
        dict(name="nvfp4 2048x4096x14336", kind="nvfp4", M=2048, N=4096, K=14336, out="bf16"),
        # a batch's tokens over many experts, some without any: gated
        dict(name="experts 48 of 32", kind="experts", M=48, N=4096, K=2048, E=32, dtype="bf16", out="bf16", gate=True),
        # a prompt's rows over a layer's experts, ragged, with room behind the last row
        dict(name="experts 6000 of 16", kind="experts", M=6000, N=4096, K=4096, E=16, dtype="bf16", out="bf16", gate=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quantize", "linear", "nvfp4", "experts"])
    dtype = rng.choice(["bf16", "f16"])
    if kind == "quantize":
        M, K = _log(rng, 1, 14336), 32 * _log(rng, 2, 448)
        M = min(M, 14336 * 4096 // K)
        return dict(kind=kind, M=M, K=K, dtype=dtype, out=rng.choice(["f32", "bf16"]) if dtype == "bf16" else "f32")
    N, K = _log(rng, 64, 28672), 32 * _log(rng, 8, 448)
    out = rng.choice(["bf16", "f16"])
    if kind == "nvfp4":
        M = _log(rng, 1, 4096)
        N = min(N, 4096 * 14336 * 4096 // (M * K))
        return dict(kind=kind, M=M, N=N, K=K, out=out)
    gate = rng.random() < 0.4
    if kind == "linear":
        M = _log(rng, 1, 4096)
        N = min(N, 4096 * 14336 * 4096 // (M * K))
        return dict(kind=kind, M=M, N=N - N % 2, K=K, dtype=dtype, out=out, gate=gate)
    E = _log(rng, 2, 64)
    M = _log(rng, 1, 6000)
    N = max(64, min(N, 4096 * 14336 * 4096 // (6000 * K), (1 << 28) // (E * K)))
    return dict(kind=kind, M=M, N=N - N % 2, K=K, E=E, dtype=dtype, out=out, gate=gate)


def _counts(case):
    """Rows of each expert: uneven, a few experts without any, and (for many rows) room behind the last."""
    rng = random.Random("%d %d %d" % (case["M"], case["E"], case["N"]))
    T, E = case["M"], case["E"]
    weight = [0.0 if e and rng.random() < 0.1 else math.exp(rng.gauss(0.0, 0.8)) for e in range(E)]
    used = T - (T // 50)
    counts = [int(used * w / sum(weight)) for w in weight]
    for _ in range(used - sum(counts)):
        counts[rng.choices(range(E), weight)[0]] += 1
    return counts


# ----------------------------------------------------------------------------------------------------- formats, in torch
def _tile(rows):
    """Scale bytes [..., R, C] as tiles [..., ceil(R/128), ceil(C/4), 512]; what pads them is 0."""
    *lead, R, C = rows.shape
    rows = torch.nn.functional.pad(rows, (0, -C % 4, 0, -R % 128))
    t = rows.view(*lead, -(-R // 128), 4, 32, -(-C // 4), 4)
    n = len(lead)
    return t.permute(*range(n), n, n + 3, n + 2, n + 1, n + 4).reshape(*lead, -(-R // 128), -(-C // 4), 512)


def _untile(tiles, R, C):
    """The scale bytes [..., R, C] of tiles."""
    *lead, rt, ct, _ = tiles.shape
    n = len(lead)
    t = tiles.view(*lead, rt, ct, 32, 4, 4).permute(*range(n), n, n + 3, n + 2, n + 1, n + 4)
    return t.reshape(*lead, rt * 128, ct * 4)[..., :R, :C]


def _code(a):
    """E2M1 codes 0..7 of magnitudes, to the nearest, ties to the even code, at most 6."""
    return ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int())


def _pack(x, scale):
    """Two codes a byte of x [R, K] / scale [R, blocks], x in blocks of K / blocks."""
    R, K = x.shape
    xs = x.view(R, scale.shape[1], -1) / scale.unsqueeze(2)
    c = (_code(xs.abs()) | ((xs < 0).int() << 3)).view(R, K // 2, 2)
    return (c[:, :, 0] | (c[:, :, 1] << 4)).to(torch.uint8)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _unpack(codes, dtype):
    """The E2M1 values [..., K] of codes [..., K / 2]."""
    table = torch.tensor(_E2M1, dtype=dtype, device=codes.device)
    c = codes.int()
    return table[torch.stack([c & 15, c >> 4], dim=-1).flatten(-2)]


def _pow2(e):
    """2 ** e in 64 bits, from its bits."""
    return ((e.long() + 1023) << 52).view(F64)


def _mx_exponent(x):
    """The scale exponents [R, K / 32] of x [R, K]: floor(log2(largest magnitude)) - 2, within [-127, 127]."""
    top = x.abs().view(x.shape[0], -1, 32).amax(2)
    return torch.where(top > 0, (torch.frexp(top)[1] - 3).clamp(-127, 127), -127)


def _mx_value(x):
    """x [R, K] (32 bits) rounded to MXFP4, as 32-bit values; every step is exact but the rounding to E2M1."""
    scale = _pow2(_mx_exponent(x)).unsqueeze(2)
    xs = x.double().view(x.shape[0], -1, 32) / scale
    table = torch.tensor(_E2M1[:8], dtype=F64, device=x.device)
    return (table[_code(xs.abs()).long()] * torch.sign(xs) * scale).view_as(x).float()


def _weights(case, gen, dev, E=None):
    """Packed weights: N(0, 0.02) with one in a thousand ten times larger."""
    N, K = case["N"] * (E or 1), case["K"]
    w = torch.randn(N, K, generator=gen, device=dev) * 0.02
    w = torch.where(torch.rand(N, K, generator=gen, device=dev) < 0.001, w * 10, w)
    if case["kind"] == "nvfp4":
        codes, scales, ts = _pack_nvfp4(w)
        return codes, _tile(scales), ts
    e = _mx_exponent(w)
    codes, scales = _pack(w, _pow2(e).float()), (e + 127).to(torch.uint8)
    if E:
        return codes.view(E, case["N"], K // 2), _tile(scales.view(E, case["N"], K // 32)), None
    return codes, _tile(scales), None


def _pack_nvfp4(x):
    ts = x.abs().amax().clamp(min=1e-30) / 2688.0
    s = (x.abs().view(x.shape[0], -1, 16).amax(2) / (6.0 * ts)).to(torch.float8_e4m3fn)
    codes = _pack(x, (s.float() * ts).clamp(min=1e-30))
    return codes, s.view(torch.uint8), ts.reshape(1)


def _acts(M, K, gen, dev):
    """Activations: N(0, 1), eight channels 50 times larger."""
    x = torch.randn(M, K, generator=gen, device=dev)
    x[:, torch.randperm(K, generator=gen, device=dev)[:8]] *= 50.0
    return x


# ------------------------------------------------------------------------------------------------------------ the inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    M, K, kind = case["M"], case["K"], case["kind"]
    s = dict(case=case, out=TYPES[case["out"]])
    if kind == "quantize":
        x = torch.randn(M, K, generator=gen, device=dev) * 0.02 if case["dtype"] == "f16" else _acts(M, K, gen, dev)
        s["x"] = x.to(TYPES[case["dtype"]])
        return s
    if kind == "nvfp4":
        s["codes_a"], s["scales_a"], s["ts_a"] = _pack_nvfp4(_acts(M, K, gen, dev))
        s["codes_w"], s["scales_w"], s["ts_w"] = _weights(case, gen, dev)
        return s
    s["x"] = _acts(M, K, gen, dev).to(TYPES[case["dtype"]])
    s["codes_w"], s["scales_w"], _ = _weights(case, gen, dev, case.get("E"))
    if kind == "experts":
        counts = _counts(case)
        ends = [sum(counts[:e]) for e in range(len(counts) + 1)]
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device=dev)
        s["most"], s["used"] = max(counts), ends[-1]
        s["y"] = torch.zeros(M, case["N"] // (2 if case["gate"] else 1), dtype=s["out"], device=dev)
    return s


# ------------------------------------------------------------------------------------------------------------- the passes
def _gated(y):
    gate, up = y[..., 0::2], y[..., 1::2]
    return gate / (1.0 + torch.exp(-gate)) * up


def _mx_weight(s):
    c = s["case"]
    w = _unpack(s["codes_w"], F32).view(*s["codes_w"].shape[:-1], -1, 32)
    e = _untile(s["scales_w"], c["N"], c["K"] // 32).int() - 127
    return (w * _pow2(e).float().unsqueeze(-1)).flatten(-2)


def _plain(s):
    c, kind = s["case"], s["case"]["kind"]
    if kind == "quantize":
        return _mx_value(s["x"].float()).to(s["out"])
    if kind == "nvfp4":
        a = _unpack(s["codes_a"], F32).view(c["M"], -1, 16) * s["scales_a"].view(torch.float8_e4m3fn).float().unsqueeze(2)
        w = _untile(s["scales_w"], c["N"], c["K"] // 16).view(torch.float8_e4m3fn).float().unsqueeze(2)
        w = _unpack(s["codes_w"], F32).view(c["N"], -1, 16) * w
        return (torch.matmul(a.flatten(1), w.flatten(1).t()) * (s["ts_a"] * s["ts_w"])).to(s["out"])
    x, w = _mx_value(s["x"].float()), _mx_weight(s)
    if kind == "linear":
        y = torch.matmul(x, w.t())
        return (_gated(y) if c["gate"] else y).to(s["out"])
    # each expert's rows, padded to the longest, in one batched product
    start, n = s["offsets"][:-1].long(), (s["offsets"][1:] - s["offsets"][:-1]).long()
    at = torch.arange(s["most"], device=x.device)
    here = at < n.unsqueeze(1)
    rows = torch.where(here, start.unsqueeze(1) + at, 0)
    y = torch.bmm(x[rows], w.transpose(1, 2))
    y = (_gated(y) if c["gate"] else y).to(s["out"])
    full = torch.zeros_like(s["y"])
    full[: s["used"]] = y[here]
    return full


def run(s):
    if not own:
        return _plain(s)
    import bit_quantization_razer_b200 as R

    c, kind = s["case"], s["case"]["kind"]
    if kind == "quantize":
        codes, scales = R.razer_quantize_mx(s["x"])
        return R.razer_dequant_mx(codes, scales, s["out"])
    if kind == "nvfp4":
        scales_a = R.razer_tile_scales(s["scales_a"])
        return R.razer_gemm_mx(s["codes_a"], scales_a, s["codes_w"], s["scales_w"], "nvfp4", s["out"], ts_a=s["ts_a"], ts_w=s["ts_w"])
    act = "silu_mul" if c["gate"] else None
    if kind == "linear":
        return R.razer_gemm_mx_online(s["x"], s["codes_w"], s["scales_w"], s["out"], act=act)
    return R.razer_gemm_mx_grouped_online(s["x"], s["offsets"], s["codes_w"], s["scales_w"], s["out"], act=act, out=s["y"])


# ------------------------------------------------------------------------------------------------------------------- work
def work(case):
    M, K = case["M"], case["K"]
    size = torch.finfo(TYPES[case["out"]]).bits // 8
    if case["kind"] == "quantize":
        return dict(bytes=M * K * (2 + 17 / 32 + size), flops=0)
    N = case["N"]
    cols = N // 2 if case.get("gate") else N
    if case["kind"] == "nvfp4":
        return dict(bytes=(M + N) * K * 9 / 16 + M * cols * size, flops=2 * M * N * K)
    if case["kind"] == "linear":
        return dict(bytes=2 * M * K + N * K * 17 / 32 + M * cols * size, flops=2 * M * N * K)
    counts = _counts(case)
    used, active = sum(counts), sum(n > 0 for n in counts)
    return dict(bytes=2 * used * K + active * N * K * 17 / 32 + used * cols * size, flops=2 * used * N * K)


# ------------------------------------------------------------------------------------------- the definition, in 64 bits
def _exact_grid(a):
    """The nearest E2M1 value of a >= 0: steps of 0.5 below 2, of 1 below 4, of 2 above, ties to the even multiple."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(F64)
    return (torch.round(a / step) * step).clamp(max=6.0)


def _exact_mx(x):
    v = x.double().unflatten(1, (-1, 32))
    top = v.abs().amax(2, keepdim=True)
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140)))
    e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e))
    scale = torch.exp2((e - 2).clamp(-127, 127))
    return (torch.copysign(_exact_grid(v.abs() / scale), v) * scale).flatten(1)


def _exact_values(codes, scale):
    """Values [..., K] of codes [..., K / 2], scale [..., K / block] in 64 bits."""
    lo, hi = codes & 15, codes >> 4
    c = torch.stack([lo, hi], -1).flatten(-2).to(F64)
    m, e = c % 2, torch.div(c % 8, 2, rounding_mode="floor")
    mag = torch.where(e == 0, m * 0.5, torch.exp2(e - 1) * (1 + m * 0.5))
    v = torch.where(c >= 8, -mag, mag)
    return (v.unflatten(-1, (scale.shape[-1], -1)) * scale.unsqueeze(-1)).flatten(-2)


def _exact_rows(tiles, R, C):
    """Scale bytes [..., R, C] out of tiles, by the byte's place."""
    r = torch.arange(R, device=tiles.device).unsqueeze(1)
    c = torch.arange(C, device=tiles.device).unsqueeze(0)
    return tiles[..., r // 128, c // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4]


def _exact_e4m3(b):
    b = b.to(F64)
    m, e = b % 8, torch.div(b, 8, rounding_mode="floor")
    return torch.where(e == 0, m * 2.0 ** -9, torch.exp2(e - 7) * (1 + m / 8))


def exact(case, seed):
    s = prepare(case, seed)
    M, K, kind = case["M"], case["K"], case["kind"]
    if kind == "quantize":
        return _exact_mx(s["x"])
    N = case["N"]
    if kind == "nvfp4":
        a = _exact_values(s["codes_a"], _exact_e4m3(s["scales_a"]))
        w = _exact_values(s["codes_w"], _exact_e4m3(_exact_rows(s["scales_w"], N, K // 16)))
        return a @ w.T * (s["ts_a"].double() * s["ts_w"].double())
    x = _exact_mx(s["x"])

    def product(x, codes, tiles):
        y = x @ _exact_values(codes, torch.exp2(_exact_rows(tiles, N, K // 32).to(F64) - 127)).T
        return y[:, 0::2] * torch.sigmoid(y[:, 0::2]) * y[:, 1::2] if case["gate"] else y

    if kind == "linear":
        return product(x, s["codes_w"], s["scales_w"])
    y = torch.zeros(s["y"].shape, dtype=F64, device=x.device)
    ends = s["offsets"].tolist()
    for e in range(case["E"]):
        if ends[e + 1] > ends[e]:
            y[ends[e]:ends[e + 1]] = product(x[ends[e]:ends[e + 1]], s["codes_w"][e], s["scales_w"][e])
    return y
