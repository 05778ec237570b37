"""The microscaled 4-bit operators on the GPU against their plain 64-bit forms:
bit-exact where they write codes, scales or decoded values; the products
within the bound of fp32 accumulation (mx_reference.product) and half a step
of the output type."""
import threading

import numpy as np
import pytest
import torch

import bit_quantization_razer_b200 as R
from tests import mx_reference as ref
from tests.gpu_helpers import cuda

pytestmark = [pytest.mark.gpu, cuda]
DEV = "cuda:0"


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a
    return t.to(DEV) if dtype is None else t.to(DEV, dtype)


def matrix(M, K, dtype, seed, spread=3.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * np.exp(spread * rng.standard_normal((M, 1)))
    return torch.from_numpy(x).to(dtype)


def offsets_of(counts, first=0):
    return [first + int(sum(counts[:e])) for e in range(len(counts) + 1)]


# ------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (129, 96), (40, 256), (5, 1024), (33, 1312), (300, 4128)])
def test_quantize_and_decode_are_exact(M, K, dtype):
    x = matrix(M, K, dtype, seed=M + K)
    x[0, :32] = 0
    if M > 2:
        x[1, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 0.0]).to(dtype)
        x[1, 16:32] = 4.0
        x[2, :32] = torch.finfo(dtype).max  # the largest values, and subnormals beside normal ones
        x[2, 32:64] = torch.finfo(dtype).tiny / 4
    codes, scales = R.razer_quantize_mx(dev(x))
    rc, rs = ref.quantize(x.double().numpy())
    assert np.array_equal(ref.untile(scales.cpu().numpy(), M, K // 32), rs)
    assert np.array_equal(ref.unpack(codes.cpu().numpy()), rc)
    if K % 128:  # what pads a tile's row is 0
        assert not ref.untile(scales.cpu().numpy(), M, -(-K // 128) * 4)[:, K // 32:].any()
    v = ref.values(codes.cpu().numpy(), rs, "mxfp4")
    for out in (torch.float32, torch.bfloat16, torch.float16):
        got = R.razer_dequant_mx(codes, scales, out)
        want = torch.from_numpy(v).to(torch.float32).to(out)  # exact in fp32, one rounding
        same = (got.cpu() == want) | (torch.isnan(got.cpu()) & torch.isnan(want))
        assert same.all()


def test_quantize_nan_and_infinity_blocks():
    for dtype in (torch.bfloat16, torch.float16):
        x = matrix(6, 128, dtype, seed=3, spread=0.0)
        x[0, 5], x[1, 40], x[2, 127], x[3, 64] = float("nan"), float("inf"), float("-inf"), float("nan")
        codes, scales = R.razer_quantize_mx(dev(x))
        rc, rs = ref.quantize(x.double().numpy())
        assert np.array_equal(ref.untile(scales.cpu().numpy(), 6, 4), rs)
        assert np.array_equal(ref.unpack(codes.cpu().numpy()), rc)
        out = R.razer_dequant_mx(codes, scales).cpu()
        bad = torch.from_numpy(np.repeat(rs == 255, 32, axis=1))
        assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()


def test_quantize_every_bf16_magnitude():
    # every finite bf16 pattern, each next to one element that sets the scale
    bits = torch.arange(0x7F80, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16).repeat(2)
    v[0x7F80:] *= -1
    x = torch.zeros(v.numel(), 32, dtype=torch.bfloat16)
    x[:, 3] = v
    x[:, 9] = (v.float() * 3.0).clamp(-3e38, 3e38).to(torch.bfloat16)
    codes, scales = R.razer_quantize_mx(dev(x))
    rc, rs = ref.quantize(x.double().numpy())
    assert np.array_equal(ref.untile(scales.cpu().numpy(), x.shape[0], 1), rs)
    assert np.array_equal(ref.unpack(codes.cpu().numpy()), rc)


@pytest.mark.parametrize("counts,first,tail", [([5, 0, 130, 1, 128, 21], 3, 7), ([0, 0, 4], 0, 0), ([1], 0, 0), ([0, 0], 2, 5),
                                               ([127, 129, 1, 1, 1, 255, 256, 0], 0, 1)])
def test_quantize_groups(counts, first, tail):
    K, off = 160, offsets_of(counts, first)
    T = off[-1] + tail
    x = matrix(T, K, torch.bfloat16, seed=T)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    codes = torch.full((T, K // 2), 0xA5, dtype=torch.uint8, device=DEV)
    scales = torch.full(R.razer_scale_tiles_shape(T, K, "mxfp4", len(counts)), 0xA5, dtype=torch.uint8, device=DEV)
    R.razer_quantize_mx(dev(x), o, codes=codes, scales=scales)
    rc, rs = ref.quantize(x.double().numpy())
    s = slice(off[0], off[-1])
    assert np.array_equal(ref.unpack(codes.cpu().numpy())[s], rc[s])
    assert (codes[: off[0]] == 0xA5).all() and (codes[off[-1]:] == 0xA5).all()  # rows of no group stay
    assert np.array_equal(ref.untile(scales.cpu().numpy(), T, K // 32, off)[s], rs[s])
    out = torch.full((T, K), -7.0, device=DEV)
    R.razer_dequant_mx(codes, scales, offsets=o, out=out)
    want = ref.values(codes.cpu().numpy(), rs, "mxfp4")
    assert np.array_equal(out.cpu().numpy()[s], want[s]) and (out[: off[0]] == -7).all() and (out[off[-1]:] == -7).all()
    # the same rows tiled from row-major scales
    tiles = R.razer_tile_scales(dev(rs), o)
    assert np.array_equal(ref.untile(tiles.cpu().numpy(), T, K // 32, off)[s], rs[s])


@pytest.mark.parametrize("R_,C", [(1, 1), (128, 4), (130, 10), (257, 16), (64, 33), (300, 128), (1000, 7)])
def test_tile_scales(R_, C):
    rng = np.random.default_rng(R_ * C)
    rows = rng.integers(0, 256, (3, R_, C)).astype(np.uint8)
    one = R.razer_tile_scales(dev(rows[0]))
    want = ref.tile(rows[0])
    assert np.array_equal(one.cpu().numpy(), want)
    assert np.array_equal(R.razer_tile_scales(dev(rows))[2].cpu().numpy(), ref.tile(rows[2]))
    # rows that start at any byte
    buf = dev(np.concatenate([np.zeros(3, np.uint8), rows[0].reshape(-1)]))
    out = torch.empty_like(one)
    L = R.load()
    assert L.razer_tile_scales(buf.data_ptr() + 3, 1, R_, C, None, 0, out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, one)


# ------------------------------------------------------------------- products
def packed(rows, K, fmt, seed, offsets=None):
    """(codes, tiles on the device, values) of random packed rows."""
    c, s = ref.random_packed(rows, K, fmt, seed)
    return dev(c), dev(ref.tile(s, offsets)), ref.values(c, s, fmt)


def scalars(fmt, seed, E=1):
    if fmt == "mxfp4":
        return None, None
    rng = np.random.default_rng(seed)
    return (torch.tensor([0.37], device=DEV), torch.from_numpy(rng.uniform(0.01, 2.0, E).astype(np.float32)).to(DEV))


def factor(ts_a, ts_w, e=0):
    return 1.0 if ts_a is None else float(ts_a[0]) * float(ts_w[e])


SIZES = [(1, 128, 256), (8, 128, 64), (7, 40, 32), (16, 200, 96), (1, 1, 160), (33, 257, 512), (32, 128, 288), (65, 64, 1024), (64, 130, 480),
         (128, 128, 4128), (129, 300, 352), (300, 72, 640), (2, 512, 8192), (500, 600, 768),
         (200, 256, 2048), (1500, 2600, 320), (700, 6000, 1088), (100, 64, 32), (193, 33, 64), (1, 5, 32)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, fmt):
    ca, sa, a = packed(M, K, fmt, seed=M * 7 + K)
    cw, sw, w = packed(N, K, fmt, seed=N * 11 + K + 1)
    ts_a, ts_w = scalars(fmt, M)
    r, _, bound = ref.product(a, w)
    f = factor(ts_a, ts_w)
    for out in (torch.float32, torch.bfloat16):
        y = R.razer_gemm_mx(ca, sa, cw, sw, fmt, out, ts_a=ts_a, ts_w=ts_w)
        ref.check(y, r * f, bound * f)
    again = R.razer_gemm_mx(ca, sa, cw, sw, fmt, out, ts_a=ts_a, ts_w=ts_w)
    assert torch.equal(again, y)
    assert R.razer_get_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(3, 5700, 2048), (34, 5762, 2080), (2, 9590, 4096)])
def test_product_split_with_two_blocks_a_processor(M, N, K):
    # clusters that share a unit along K, more blocks than processors
    ca, sa, a = packed(M, K, "mxfp4", seed=M)
    cw, sw, w = packed(N, K, "mxfp4", seed=N)
    r, _, bound = ref.product(a, w)
    y = R.razer_gemm_mx(ca, sa, cw, sw, "mxfp4", torch.float32)
    ref.check(y, r, bound)
    assert torch.equal(R.razer_gemm_mx(ca, sa, cw, sw, "mxfp4", torch.bfloat16), y.bfloat16())
    assert R.razer_get_device_status() == 0


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(1, 128, 256), (5, 34, 96), (40, 256, 320), (130, 514, 512)])
def test_product_gated(M, N, K, fmt):
    rng = np.random.default_rng(M + N)
    c, s = ref.random_packed(M, K, fmt, M, spread=2)
    ca, sa, a = dev(c), dev(ref.tile(s)), ref.values(c, s, fmt)
    c, s = ref.random_packed(N, K, fmt, N, spread=2)
    cw, sw, w = dev(c), dev(ref.tile(s)), ref.values(c, s, fmt)
    # a scale that keeps the gates in the range where silu bends
    g = 3.0 / np.abs(a @ w.T).mean()
    ts_a, ts_w = torch.tensor([g], dtype=torch.float32, device=DEV), torch.ones(1, device=DEV)
    r, _, bound = ref.product(a, w)
    f = float(ts_a[0])
    r, bound = ref.silu_mul(r * f, bound * f)
    for out in (torch.float32, torch.float16, torch.bfloat16):
        y = R.razer_gemm_mx(ca, sa, cw, sw, fmt, out, ts_a=ts_a, ts_w=ts_w, act="silu_mul")
        assert y.shape == (M, N // 2)
        ref.check(y, r, bound)


@pytest.mark.parametrize("counts", [[70] * 40, [0] * 33 + [300] + [0] * 40 + [128, 1, 500, 90], [65, 192, 193, 64, 63]])
def test_product_grouped_many_rows_a_group(counts):
    # more groups than a warp looks up at once, empty ones between, pieces of every size
    E, N, K, off = len(counts), 136, 160, offsets_of(counts, 2)
    T = off[-1] + 3
    ca, sa, a = packed(T, K, "mxfp4", T, offsets=off)
    c, s = ref.random_packed(E * N, K, "mxfp4", E)
    w = ref.values(c, s, "mxfp4").reshape(E, N, K)
    sw = torch.stack([dev(ref.tile(x)) for x in s.reshape(E, N, -1)])
    y = torch.full((T, N), 77.0, device=DEV)
    R.razer_gemm_mx_grouped(ca, sa, torch.tensor(off, dtype=torch.int32, device=DEV), dev(c).view(E, N, K // 2), sw, out=y)
    assert (y[:2] == 77).all() and (y[off[-1]:] == 77).all()
    for e in np.flatnonzero(counts):
        r, _, bound = ref.product(a[off[e]:off[e + 1]], w[e])
        ref.check(y[off[e]:off[e + 1]], r, bound)


@pytest.mark.parametrize("counts", [[150] + [0] * 19, [1, 0, 130, 0, 0, 3, 65, 2] + [0] * 12, [7] * 64, [150] + [0] * 37, [1, 0, 130, 0, 0, 3, 65, 2] + [0] * 43,
                                    [2] * 64, [70, 40, 17, 31, 0, 1] + [0] * 40])
@pytest.mark.parametrize("gate", [False, True])
def test_grouped_online_uneven_groups(counts, gate):
    # few rows a group on average, quantized before the product and (up to 4) inside it, groups of more than one piece among them
    E, N, K, off = len(counts), 96, 544, offsets_of(counts, 1)
    T = off[-1] + 2
    x = dev(matrix(T, K, torch.bfloat16, T, 0.5))
    c, s = ref.random_packed(E * N, K, "mxfp4", E, spread=2)
    cw, sw = dev(c).view(E, N, K // 2), torch.stack([dev(ref.tile(v)) for v in s.reshape(E, N, -1)])
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    assert (R.razer_gemm_mx_grouped_workspace_size(T, K, E) == 0) == (T <= 4 * E)
    act = "silu_mul" if gate else None
    codes, tiles = R.razer_quantize_mx(x, o)
    y, z = (torch.full((T, N // 2 if gate else N), 77.0, device=DEV) for _ in range(2))
    R.razer_gemm_mx_grouped(codes, tiles, o, cw, sw, act=act, out=y)
    R.razer_gemm_mx_grouped_online(x, o, cw, sw, act=act, out=z)
    assert torch.equal(y, z) and (z[0] == 77).all() and (z[off[-1]:] == 77).all()
    a, w = ref.values(codes.cpu().numpy(), ref.untile(tiles.cpu().numpy(), T, K // 32, off), "mxfp4"), ref.values(c, s, "mxfp4").reshape(E, N, K)
    for e in np.flatnonzero(counts):
        r, _, bound = ref.product(a[off[e]:off[e + 1]], w[e])
        if gate:
            with np.errstate(over="ignore"):
                r, bound = ref.silu_mul(r, bound)
        ref.check(z[off[e]:off[e + 1]], r, bound)


def test_online_nan_reaches_its_row_only():
    for M in (5, 40):  # quantized inside the product, and before it
        x = matrix(M, 256, torch.bfloat16, 1, 0.0)
        x[2, 77] = float("nan")
        x[3, 200] = float("inf")
        cw, sw, _ = packed(130, 256, "mxfp4", 3)
        y = R.razer_gemm_mx_online(dev(x), cw, sw, torch.float32)
        bad = torch.zeros(M, dtype=torch.bool, device=DEV)
        bad[2:4] = True
        assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


def test_product_empty_shapes():
    K = 64
    ca, sa, _ = packed(5, K, "mxfp4", 1)
    cw, sw, _ = packed(9, K, "mxfp4", 2)
    assert R.razer_gemm_mx(ca[:0], sa[:0], cw, sw).shape == (0, 9)
    assert R.razer_gemm_mx(ca, sa, cw[:0], sw[:0]).shape == (5, 0)
    # K = 0: empty sums
    y = torch.full((5, 9), 3.0, device=DEV)
    R.razer_gemm_mx(ca[:, :0].contiguous(), sa[:, :0].contiguous(), cw[:, :0].contiguous(), sw[:, :0].contiguous(), out=y)
    assert not y.any()
    o = torch.tensor([1, 3, 4], dtype=torch.int32, device=DEV)
    y = torch.full((5, 9), 3.0, device=DEV)
    e = torch.empty
    R.razer_gemm_mx_grouped(ca[:, :0].contiguous(), e((2, 0, 512), dtype=torch.uint8, device=DEV), o,
                            e((2, 9, 0), dtype=torch.uint8, device=DEV), e((2, 1, 0, 512), dtype=torch.uint8, device=DEV), out=y)
    assert not y[1:4].any() and (y[0] == 3).all() and (y[4] == 3).all()
    assert R.razer_quantize_mx(torch.empty(0, 64, dtype=torch.float16, device=DEV))[0].shape == (0, 32)


def test_product_nan_scale_reaches_its_row_only():
    M, N, K = 40, 140, 384
    c, s = ref.random_packed(M, K, "mxfp4", 1)
    s[7, 3] = 255
    cw, sw, w = packed(N, K, "mxfp4", 2)
    s_ok = s.copy()
    s_ok[7, 3] = 127
    y = R.razer_gemm_mx(dev(c), dev(ref.tile(s)), cw, sw, out_dtype=torch.float32)
    assert torch.isnan(y[7]).all()
    r, _, bound = ref.product(ref.values(c, s_ok, "mxfp4"), w)
    keep = np.arange(M) != 7
    ref.check(y[torch.from_numpy(keep).to(DEV)], r[keep], bound[keep])
    # tile rows past the matrix may hold anything, NaN bytes too
    y2 = R.razer_gemm_mx(dev(c), dev(ref.tile(s_ok, fill=255)), cw, dev(sw.cpu().numpy()), out_dtype=torch.float32)
    ref.check(y2, r, bound)


GROUPS = [([3, 0, 1, 5], 0, 0), ([0, 0, 0], 2, 3), ([1] * 40, 1, 2), ([33, 0, 2, 64, 31], 5, 9), ([130, 260, 0, 7], 0, 4), ([0, 513], 0, 0),
          ([70, 70, 70, 0, 1, 200], 11, 30), ([700, 3, 0, 1000, 190, 193, 65], 1, 2)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("N,K,gate", [(128, 256, False), (200, 352, False), (72, 96, True), (40, 1056, False)])
@pytest.mark.parametrize("counts,first,tail", GROUPS)
def test_product_grouped(counts, first, tail, N, K, gate, fmt):
    E, off = len(counts), offsets_of(counts, first)
    T = off[-1] + tail
    rng = np.random.default_rng(T + N)
    ca, sa, a = packed(T, K, fmt, T, offsets=off)
    c, s = ref.random_packed(E * N, K, fmt, N)
    w = ref.values(c, s, fmt).reshape(E, N, K)
    cw = dev(c).view(E, N, K // 2)
    sw = torch.stack([dev(ref.tile(x)) for x in s.reshape(E, N, -1)])
    ts_a, ts_w = scalars(fmt, T, E)
    cols = N // 2 if gate else N
    y = torch.full((T, cols), 77.0, device=DEV)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    R.razer_gemm_mx_grouped(ca, sa, o, cw, sw, fmt, ts_a=ts_a, ts_w=ts_w, act="silu_mul" if gate else None, out=y)
    assert (y[: off[0]] == 77).all() and (y[off[-1]:] == 77).all()  # rows of no group stay
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        if counts[e] == 0:
            continue
        r, _, bound = ref.product(a[rows], w[e])
        f = factor(ts_a, ts_w, e)
        r, bound = r * f, bound * f
        if gate:
            with np.errstate(over="ignore"):
                r, bound = ref.silu_mul(r, bound)
        ref.check(y[rows], r, bound)
    assert R.razer_get_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (5, 130, 96), (16, 512, 4096), (17, 64, 1056), (100, 320, 640), (300, 260, 288)])
def test_online_equals_the_two_calls(M, N, K, dtype):
    x = dev(matrix(M, K, dtype, seed=M, spread=0.5))
    cw, sw, _ = packed(N, K, "mxfp4", N)
    codes, scales = R.razer_quantize_mx(x)
    for act in (None, "silu_mul"):
        want = R.razer_gemm_mx(codes, scales, cw, sw, act=act)
        assert torch.equal(R.razer_gemm_mx_online(x, cw, sw, act=act), want)
    counts = [M // 3, 0, M - M // 3]
    o = torch.tensor(offsets_of(counts), dtype=torch.int32, device=DEV)
    cg, sg = torch.stack([cw, cw.flip(0), cw]), torch.stack([sw] * 3)
    codes, scales = R.razer_quantize_mx(x, o)
    want = R.razer_gemm_mx_grouped(codes, scales, o, cg, sg)
    assert torch.equal(R.razer_gemm_mx_grouped_online(x, o, cg, sg), want)


def test_nvfp4_tensors_of_the_quantizers():
    # packed by the framework's NVFP4 quantizers, multiplied as they are
    M, N, K = 70, 192, 512
    x, w = matrix(M, K, torch.bfloat16, 1, 0.0), matrix(N, K, torch.float16, 2, 0.0) * 0.02
    ca, sa, ta, _ = R.razer_quantize_acts(dev(x), fmt="nvfp4", hist=False)
    cw, sw, tw = R.razer_quantize_weights(dev(w), "nvfp4")
    y = R.razer_gemm_mx(ca, R.razer_tile_scales(sa), cw, R.razer_tile_scales(sw), "nvfp4", torch.float32, ts_a=ta, ts_w=tw)
    f = float(ta[0]) * float(tw[0])
    r, _, bound = ref.product(ref.values(ca.cpu().numpy(), sa.cpu().numpy(), "nvfp4"), ref.values(cw.cpu().numpy(), sw.cpu().numpy(), "nvfp4"))
    ref.check(y, r * f, bound * f)
    # the decode-and-multiply path gives the same product within both paths' bounds
    z = R.razer_gemm_w4a4(ca, sa, ta, cw, sw, tw, "nvfp4", "nvfp4", torch.float32)
    ref.check(z, r * f, bound * f * 4)


def test_an_experts_layer():
    """The operators as a layer of experts uses them: gated pair, packing in between, projection back."""
    T, D, H, E = 90, 256, 192, 5
    counts, first = [20, 0, 1, 60, 6], 0
    off = offsets_of(counts)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    x = dev(matrix(T, D, torch.bfloat16, 5, 0.3))
    wu = dev(matrix(E * 2 * H, D, torch.bfloat16, 6, 0.0) * 0.1)
    wd = dev(matrix(E * D, H, torch.bfloat16, 7, 0.0) * 0.1)
    def pack(w, n):
        c, s = zip(*[R.razer_quantize_mx(m) for m in w.view(E, n, -1)])
        return torch.stack(c), torch.stack(s)
    cu, su = pack(wu, 2 * H)
    cd, sd = pack(wd, D)
    h = R.razer_gemm_mx_grouped_online(x, o, cu, su, act="silu_mul")
    y = R.razer_gemm_mx_grouped_online(h, o, cd, sd)
    q = lambda t: ref.values(*_host(R.razer_quantize_mx(t)), "mxfp4")
    def _host(p):
        return p[0].cpu().numpy(), ref.untile(p[1].cpu().numpy(), p[0].shape[0], p[0].shape[1] // 16)
    xv, hv = q(x), q(h)
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        if counts[e] == 0:
            continue
        r, _, b = ref.product(xv[rows], q(wu.view(E, 2 * H, D)[e]))
        ref.check(h[rows], *ref.silu_mul(r, b))
        r, _, b = ref.product(hv[rows], q(wd.view(E, D, H)[e]))
        ref.check(y[rows], r, b)
    assert not y[off[-1]:].any()


# ------------------------------------------------------- streams, graphs, rules
def test_side_stream_and_graph_replay():
    M, N, K = 24, 256, 512
    cw, sw, _ = packed(N, K, "mxfp4", 1)
    x = dev(matrix(M, K, torch.bfloat16, 2, 0.0))
    x2 = dev(matrix(M, K, torch.bfloat16, 3, 0.0))
    want, want2 = R.razer_gemm_mx_online(x, cw, sw), R.razer_gemm_mx_online(x2, cw, sw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y = R.razer_gemm_mx_online(x, cw, sw)
    other = R.razer_gemm_mx_online(x2, cw, sw, stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(other, want2)
    buf, o = x.clone(), torch.tensor([0, 4, 4, 24], dtype=torch.int32, device=DEV)
    cg, sg = torch.stack([cw] * 3), torch.stack([sw] * 3)
    out, grouped = torch.empty_like(want), torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        R.razer_gemm_mx_online(buf, cw, sw, out=out)
        R.razer_gemm_mx_grouped_online(buf, o, cg, sg, out=grouped)
    for src, w in ((x2, want2), (x, want)):
        buf.copy_(src)
        o.copy_(torch.tensor([0, 9, 20, 24], dtype=torch.int32))  # other groups than at capture
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w) and torch.equal(grouped, w)


def test_offsets_that_break_the_rules_are_reported():
    # brought into range on the device: nothing is read or written outside
    T, N, K = 40, 64, 128
    x = dev(matrix(T, K, torch.bfloat16, 4, 0.0))
    c, s = ref.random_packed(2 * N, K, "mxfp4", 9)
    cw, sw = dev(c).view(2, N, K // 2), torch.stack([dev(ref.tile(v)) for v in s.reshape(2, N, -1)])
    for off in ([0, 30, 20], [-5, 10, 40], [0, 10, 41]):
        y = torch.zeros(T, N, device=DEV)
        R.razer_gemm_mx_grouped_online(x, torch.tensor(off, dtype=torch.int32, device=DEV), cw, sw, out=y)
        assert R.razer_get_device_status() == 1
    R.razer_gemm_mx_grouped_online(x, torch.tensor([0, 10, 40], dtype=torch.int32, device=DEV), cw, sw, out=y)
    assert R.razer_get_device_status() == 0


@pytest.mark.parametrize("M", [8, 300])
def test_stalled_pipeline_reports_a_timeout_and_recovers(M):
    N, K = 128, 2048
    ca, sa, a = packed(M, K, "mxfp4", 1)
    cw, sw, w = packed(N, K, "mxfp4", 2)
    prev = R.razer_debug_set_fault_injection(True)
    try:
        R.razer_gemm_mx(ca, sa, cw, sw)
        assert R.razer_get_device_status() == 7
        if M <= 16:
            R.razer_gemm_mx_online(dev(matrix(M, K, torch.bfloat16, 3, 0.0)), cw, sw)
            assert R.razer_get_device_status() == 7
    finally:
        R.razer_debug_set_fault_injection(prev)
    y = R.razer_gemm_mx(ca, sa, cw, sw, out_dtype=torch.float32)
    r, _, bound = ref.product(a, w)
    ref.check(y, r, bound)
    assert R.razer_get_device_status() == 0


def test_stream_argument_owns_what_it_allocates():
    # the workspace of an online call on another stream must not be handed to
    # work of the current one before that stream is done with it
    M, N, K = 200, 4096, 4096
    cw, sw, _ = packed(N, K, "mxfp4", 1)
    x = dev(matrix(M, K, torch.bfloat16, 2, 0.0))
    want = R.razer_gemm_mx_online(x, cw, sw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        y = R.razer_gemm_mx_online(x, cw, sw, stream=side)
        junk = torch.full((R.razer_workspace_size(R.RAZER_OP_GEMM_MX_ONLINE, M, N, K),), 255, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        del junk, y


def test_first_call_of_a_size_in_a_capture():
    # nothing a call does for the first time (attributes, occupancy) is barred while capturing
    M, N, K = 130, 258, 96
    ca, sa, a = packed(M, K, "nvfp4", 1)
    cw, sw, w = packed(N, K, "nvfp4", 2)
    one, y = torch.ones(1, device=DEV), torch.zeros(M, N // 2, dtype=torch.float16, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        R.razer_gemm_mx(ca, sa, cw, sw, "nvfp4", ts_a=one, ts_w=one, act="silu_mul", out=y)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, R.razer_gemm_mx(ca, sa, cw, sw, "nvfp4", torch.float16, ts_a=one, ts_w=one, act="silu_mul"))


@pytest.mark.parametrize("E", [255, 256, 300])
def test_hundreds_of_groups(E):
    # more groups than the quantizer keeps in shared memory
    N, K = 72, 96
    counts = [(5 * e) % 4 for e in range(E)]
    counts[E // 2] = 140
    off = offsets_of(counts, 1)
    T = off[-1] + 3
    x = matrix(T, K, torch.bfloat16, E, 0.0)
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    codes, tiles = R.razer_quantize_mx(dev(x), o)
    rc, rs = ref.quantize(x.double().numpy())
    s = slice(off[0], off[-1])
    assert np.array_equal(ref.unpack(codes.cpu().numpy())[s], rc[s])
    assert np.array_equal(ref.untile(tiles.cpu().numpy(), T, K // 32, off)[s], rs[s])
    c, ws = ref.random_packed(E * N, K, "mxfp4", E, spread=2)
    cw, sw = dev(c).view(E, N, K // 2), torch.stack([dev(ref.tile(v)) for v in ws.reshape(E, N, -1)])
    y = R.razer_gemm_mx_grouped(codes, tiles, o, cw, sw, out_dtype=torch.float32)
    assert torch.equal(R.razer_gemm_mx_grouped_online(dev(x), o, cw, sw, torch.float32), y) and not y[0].any() and not y[off[-1]:].any()
    a, w = ref.values(codes.cpu().numpy(), rs, "mxfp4"), ref.values(c, ws, "mxfp4").reshape(E, N, K)
    for e in np.flatnonzero(counts):
        r, _, bound = ref.product(a[off[e]:off[e + 1]], w[e])
        ref.check(y[off[e]:off[e + 1]], r, bound)


def test_calls_of_two_host_threads():
    N, K = 520, 1024
    cw, sw, _ = packed(N, K, "mxfp4", 1)
    xs = [dev(matrix(M, K, torch.bfloat16, M, 0.0)) for M in (3, 200)]
    want = [R.razer_gemm_mx_online(x, cw, sw) for x in xs]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def calls(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(50):
                got[i].append(R.razer_gemm_mx_online(xs[i], cw, sw, stream=stream))
            stream.synchronize()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for i in range(2):
        assert len(got[i]) == 50 and all(torch.equal(y, want[i]) for y in got[i])


def test_captured_grouped_call_with_every_row_in_one_group():
    # the kernel is chosen by the rows a group on average, at capture; the offsets may then be any
    E, N, K, T = 40, 136, 288, 400
    c, ws = ref.random_packed(E * N, K, "mxfp4", E, spread=2)
    cw, sw = dev(c).view(E, N, K // 2), torch.stack([dev(ref.tile(v)) for v in ws.reshape(E, N, -1)])
    x = matrix(T, K, torch.bfloat16, T, 0.0)
    o = torch.tensor([i * 10 for i in range(E + 1)], dtype=torch.int32, device=DEV)
    xd, y = dev(x), torch.zeros(T, N, device=DEV)
    R.razer_gemm_mx_grouped_online(xd, o, cw, sw, out=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        R.razer_gemm_mx_grouped_online(xd, o, cw, sw, out=y)
    rc, rs = ref.quantize(x.double().numpy())
    codes, tiles = R.razer_quantize_mx(xd)
    a = ref.values(codes.cpu().numpy(), rs, "mxfp4")
    w = ref.values(c, ws, "mxfp4").reshape(E, N, K)
    for e in (0, 17, E - 1):
        o.copy_(torch.tensor([0 if i <= e else T for i in range(E + 1)], dtype=torch.int32))
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        r, _, bound = ref.product(a, w[e])
        ref.check(y, r, bound)
    assert R.razer_get_device_status() == 0
