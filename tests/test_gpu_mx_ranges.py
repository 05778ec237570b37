"""The microscaled products at the ends of their ranges (gates whose exponential
nears the end of fp32's, scale bytes 0 and 254, sums beyond fp32), and forms of
their outputs: f16, and gated ones of sums joined over clusters."""
import numpy as np
import pytest
import torch

import bit_quantization_razer_b200 as R
from tests import mx_reference as ref
from tests.gpu_helpers import cuda

pytestmark = [pytest.mark.gpu, cuda]
DEV = "cuda:0"


def dev(a):
    return (torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a).to(DEV)


def pack(codes):
    """codes [R, K] 0..15 -> bytes."""
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


@pytest.mark.parametrize("M", [6, 130])  # both kernels
def test_gates_to_the_end_of_the_exponential(M):
    # Block 0 of a row makes the gate, exact multiples of 1/16 from -96 to 96; block 1 makes up projections of
    # 2^110 and more, beside which silu(-88.7) is not small.
    rng = np.random.default_rng(M)
    J = 66
    a, w = np.zeros((M, 64), np.int64), np.zeros((2 * J, 64), np.int64)
    a[:, :32] = 7  # 6, and in some places less
    for i in range(M):
        at = rng.permutation(32)
        a[i, at[: (0, 8, 7, 8, 12, 20)[i % 6]]] = 6  # 4: the gate 1 nearer to 0 for each
        if i >= 6:
            a[i, at[-1]] = rng.integers(0, 8)
    a[:, 32:], w[1::2, 32:] = rng.integers(0, 16, (M, 32)), rng.integers(0, 16, (J, 32))
    w[0::2, :32] = np.array([0xE, 0xE, 0xE, 0x6, 0xC, 0xA])[np.arange(J) % 6, None]  # -4, -4, -4, 4, -2, -1
    sa, sw = np.full((M, 2), 127 - 3, np.uint8), np.full((2 * J, 2), 127, np.uint8)
    sa[:, 1], sw[1::2, 1] = 127 + 60, 127 + 50
    y = ref.values(pack(a), sa, "mxfp4") @ ref.values(pack(w), sw, "mxfp4").T  # exact, in fp32 too
    g, u = y[:, 0::2], y[:, 1::2]
    assert (g == np.round(16 * g) / 16).all() and g.min() == -96 and ((g < -87.5) & (g > -88.7)).sum() >= 3
    finite = -g < 128 * np.log(2)  # exp(-g) within fp32's range: else 0
    r = np.where(finite, g / (1 + np.exp(np.where(finite, -g, 0))), 0) * u
    x = (dev(pack(a)), dev(ref.tile(sa)), dev(pack(w)), dev(ref.tile(sw)))
    for out, err in ((torch.bfloat16, 6e-6), (torch.float16, 6e-6), (torch.float32, 8 * 2.0 ** -23)):
        got = R.razer_gemm_mx(*x, out_dtype=out, act="silu_mul")
        ref.check(got, r, err * np.abs(r))
    assert R.razer_get_device_status() == 0


def packed_with(rows, K, seed, scales, codes=None):
    """Random MXFP4 rows whose scale bytes are drawn from `scales` -> (codes, tiles on the device, values)."""
    rng = np.random.default_rng(seed)
    c = pack(rng.integers(0, 16, (rows, K)) if codes is None else codes(rng, (rows, K)))
    s = rng.choice(np.asarray(scales, np.uint8), (rows, K // 32))
    return dev(c), dev(ref.tile(s)), ref.values(c, s, "mxfp4")


@pytest.mark.parametrize("M,N,K", [(5, 200, 288), (70, 130, 4096), (200, 264, 544)])
def test_scales_at_both_ends_of_e8m0(M, N, K):
    # 2^-127 against 2^127: every product is near 1, and so are the sums
    for lo, hi in (([0], [254]), ([254], [0]), ([0, 1, 2], [252, 253, 254])):
        ca, sa, a = packed_with(M, K, M, lo)
        cw, sw, w = packed_with(N, K, N + 1, hi)
        r, _, bound = ref.product(a, w)
        for out in (torch.float32, torch.float16, torch.bfloat16):
            ref.check(R.razer_gemm_mx(ca, sa, cw, sw, out_dtype=out), r, bound)
    assert R.razer_get_device_status() == 0


@pytest.mark.parametrize("M", [5, 200])
def test_blocks_of_zeros_beside_live_ones(M):
    # what the quantizer writes for a block of zeros: byte 0, codes 0, here also -0
    N, K = 136, 544
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16)
    x[:, 64:128] = 0
    x[1:3, :] = 0
    x[2, 5::7] = -0.0
    codes, tiles = R.razer_quantize_mx(dev(x))
    rc, rs = ref.quantize(x.double().numpy())
    assert (rs[:, 2:4] == 0).all() and (rs[1:3] == 0).all()
    cw, sw, w = packed_with(N, K, 3, range(117, 138))
    r, _, bound = ref.product(ref.values(pack(rc), rs, "mxfp4"), w)
    for y in (R.razer_gemm_mx(codes, tiles, cw, sw, out_dtype=torch.float32), R.razer_gemm_mx_online(dev(x), cw, sw, torch.float32)):
        ref.check(y, r, bound)
        assert not y[1:3].any()


@pytest.mark.parametrize("M", [5, 200])
def test_sums_beyond_fp32(M):
    # 2^127 squared: infinite, of the sums' sign, in the rows and columns that reach it and in no others
    N, K = 72, 96
    plus = lambda rng, shape: rng.integers(1, 8, shape)
    ca, sa, a = packed_with(M, K, M, [127], plus)
    cw, sw, w = packed_with(N, K, N, [127], plus)
    c, s = ca.cpu().numpy(), ref.untile(sa.cpu().numpy(), M, K // 32)
    s[3] = 254
    a = ref.values(c, s, "mxfp4")
    t = ref.untile(sw.cpu().numpy(), N, K // 32)
    t[7] = t[40] = 254
    v = cw.cpu().numpy()
    v[40] |= 0x88  # negative
    w = ref.values(v, t, "mxfp4")
    r, _, bound = ref.product(a, w)
    for out in (torch.float32, torch.bfloat16, torch.float16):
        y = R.razer_gemm_mx(ca, dev(ref.tile(s)), dev(v), dev(ref.tile(t)), out_dtype=out).double().cpu().numpy()
        assert y[3, 7] == np.inf and y[3, 40] == -np.inf
        assert not np.isnan(y).any()
        far = np.abs(r) + bound >= torch.finfo(out).max
        assert (np.sign(y[far]) == np.sign(r[far])).all()
        ref.check(torch.from_numpy(y).to(out), r, bound)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(1, 128, 256), (7, 41, 96), (40, 257, 512), (3, 258, 4096), (65, 64, 1024), (129, 300, 352), (128, 258, 4128),
                                   (500, 601, 768)])
def test_f16_outputs(M, N, K, fmt):
    # scaled so that the sums keep to f16's range; N even and odd: outputs stored in pairs and alone
    rng = np.random.default_rng(M + N)
    (ca, sca), (cw, scw) = (ref.random_packed(n, K, fmt, rng.integers(1 << 30), spread=2) for n in (M, N))
    a, w = ref.values(ca, sca, fmt), ref.values(cw, scw, fmt)
    r, _, bound = ref.product(a, w)
    ts = np.float32(100.0 / np.abs(r).mean())
    y = R.razer_gemm_mx(dev(ca), dev(ref.tile(sca)), dev(cw), dev(ref.tile(scw)), fmt, torch.float16, ts_a=torch.tensor([ts], device=DEV),
                        ts_w=torch.ones(1, device=DEV))
    ref.check(y, r * float(ts), bound * float(ts))
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("M,N,K", [(3, 258, 4096), (20, 130, 8224), (64, 514, 4128), (128, 258, 4128), (100, 514, 8192)])
def test_gated_outputs_of_sums_joined_over_clusters(M, N, K, fmt):
    # few units of long K: both kernels split K, and gate and up meet after their sums are joined
    rng = np.random.default_rng(M + N + K)
    (ca, sca), (cw, scw) = (ref.random_packed(n, K, fmt, rng.integers(1 << 30), spread=2) for n in (M, N))
    a, w = ref.values(ca, sca, fmt), ref.values(cw, scw, fmt)
    r, _, bound = ref.product(a, w)
    ts = np.float32(3.0 / np.abs(r).mean())  # gates where silu bends
    r, bound = ref.silu_mul(r * float(ts), bound * float(ts))
    for out in (torch.float32, torch.float16, torch.bfloat16):
        y = R.razer_gemm_mx(dev(ca), dev(ref.tile(sca)), dev(cw), dev(ref.tile(scw)), fmt, out, ts_a=torch.tensor([ts], device=DEV),
                            ts_w=torch.ones(1, device=DEV), act="silu_mul")
        ref.check(y, r, bound + (5e-6 * np.abs(r) if out != torch.float32 else 0.0))
    assert R.razer_get_device_status() == 0
