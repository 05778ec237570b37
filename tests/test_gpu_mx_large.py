"""The microscaled 4-bit operators past 2^31: codes of more than 2^31 bytes,
outputs of more than 2^31 elements, checked on sampled rows."""
import numpy as np
import pytest
import torch

import bit_quantization_razer_b200 as R
from tests import mx_reference as ref
from tests.gpu_helpers import cuda

pytestmark = [pytest.mark.gpu, cuda]
DEV = "cuda:0"


def test_quantize_and_product_past_2_31():
    M, N, K = 540_003, 4096, 8192
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV).normal_(0.0, 1.0, generator=g)
    w = torch.empty(N, K, dtype=torch.bfloat16, device=DEV).normal_(0.0, 0.02, generator=g)
    codes, scales = R.razer_quantize_mx(x)
    assert codes.numel() > 1 << 31
    rows = np.unique(np.concatenate([[0, M - 1, (1 << 31) * 2 // K, (1 << 31) * 2 // K + 1, (1 << 31) // N, (1 << 31) // N + 1],
                                     np.random.default_rng(0).integers(0, M, 26)]))
    at = torch.from_numpy(rows).to(DEV)
    rc, rs = ref.quantize(x[at].double().cpu().numpy())
    assert np.array_equal(ref.unpack(codes[at].cpu().numpy()), rc)
    c = torch.arange(K // 32, device=DEV)
    got = scales[at[:, None] // 128, c[None] // 4, ((at % 32) * 16 + at % 128 // 32 * 4)[:, None] + c[None] % 4]
    assert np.array_equal(got.cpu().numpy(), rs)
    back = R.razer_dequant_mx(codes, scales, torch.bfloat16)  # exact in bf16
    a = ref.values(codes[at].cpu().numpy(), rs, "mxfp4")
    assert np.array_equal(back[at].double().cpu().numpy(), a)
    del x, back
    cw, sw = R.razer_quantize_mx(w)
    wv = ref.values(cw.cpu().numpy(), ref.untile(sw.cpu().numpy(), N, K // 32), "mxfp4")
    y = R.razer_gemm_mx(codes, scales, cw, sw)
    assert y.numel() > 1 << 31
    r, _, bound = ref.product(a, wv)
    ref.check(y[at], r, bound)
    # the same rows as two groups that meet near the end
    off = [3, M - 130, M - 1]
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    tiles = torch.zeros(R.razer_scale_tiles_shape(M, K, "mxfp4", 2), dtype=torch.uint8, device=DEV)
    flat = scales.view(-1, scales.shape[1], 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, scales.shape[1] * 4)[:M, :K // 32].contiguous()
    R.razer_tile_scales(flat, o, out=tiles)
    y2 = torch.zeros_like(y)
    R.razer_gemm_mx_grouped(codes, tiles, o, torch.stack([cw, cw]), torch.stack([sw, sw]), out=y2)
    inside = torch.from_numpy(rows[(rows >= 3) & (rows < M - 1)]).to(DEV)
    assert torch.equal(y2[inside], y[inside]) and not y2[:3].any() and not y2[M - 1].any()
    assert torch.equal(y2[M - 200:M - 1], y[M - 200:M - 1])


def bytes_of(shape, lo, hi, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(lo, hi, shape, dtype=torch.uint8, device=DEV, generator=g)


def dev(a):
    return torch.from_numpy(a).to(DEV)


def test_weight_rows_near_2_31():
    # the last tile of 128 rows ends at 2^31
    M, N, K = 2, (1 << 31) - 1, 32
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB of device memory")
    cw, sw = bytes_of((N, K // 2), 0, 256, 1), bytes_of(R.razer_scale_tiles_shape(N, K), 120, 135, 2)
    sw[:, 0].view(-1, 32, 4, 4)[..., 1:] = 0  # what lies past K / 32 = 1 scale
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(3)).to(DEV, torch.bfloat16)
    ca, sa = R.razer_quantize_mx(x)
    y = R.razer_gemm_mx(ca, sa, cw, sw)
    rows = np.unique(np.concatenate([np.arange(200), np.arange(N - 400, N), np.random.default_rng(0).integers(0, N, 200)]))
    at = torch.from_numpy(rows).to(DEV)
    w = ref.values(cw[at].cpu().numpy(), sw[at // 128, 0, (at % 32) * 16 + at % 128 // 32 * 4].cpu().numpy()[:, None], "mxfp4")
    a = ref.values(ca.cpu().numpy(), ref.untile(sa.cpu().numpy(), M, 1), "mxfp4")
    r, _, bound = ref.product(a, w)
    ref.check(y[:, at], r, bound)
    assert R.razer_get_device_status() == 0
    z = torch.full_like(y, 7.0)
    R.razer_gemm_mx_online(x, cw, sw, out=z)
    assert torch.equal(y[0], z[0]) and torch.equal(y[1], z[1])


def test_row_length_near_2_31():
    # few blocks are not zero, the first and the last of a row among them: every sum is exact
    M, N, K = 2, 3, (1 << 31) - 32
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB of device memory")
    C = K // 32
    blocks = [0, 7, C // 2, C - 9, C - 1]
    rng = np.random.default_rng(7)
    ac, wc = (rng.integers(0, 256, (n, len(blocks), 16), dtype=np.uint8) for n in (M, N))

    def matrix(codes):
        c = torch.zeros(len(codes), K // 2, dtype=torch.uint8, device=DEV)
        t = torch.full(R.razer_scale_tiles_shape(len(codes), K), 127, dtype=torch.uint8, device=DEV)
        t[:, -1].view(-1, 32, 4, 4)[..., 3] = 0  # what lies past the last scale
        for i, b in enumerate(blocks):
            c[:, 16 * b:16 * b + 16] = torch.from_numpy(codes[:, i]).to(DEV)
        return c, t

    (ca, sa), (cw, sw) = matrix(ac), matrix(wc)
    a, w = (ref.E2M1[ref.unpack(v)].reshape(len(v), -1) for v in (ac, wc))
    want = torch.from_numpy(a @ w.T)  # multiples of 1/4 below 2^13
    y = R.razer_gemm_mx(ca, sa, cw, sw, out_dtype=torch.float32)
    assert torch.equal(y.double().cpu(), want)
    del ca, sa
    # quantized in the product: a block's largest magnitude 6 or 4 leaves its values as they are
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    ac[:, :, 0] = 0x77
    a = ref.E2M1[ref.unpack(ac)].reshape(M, len(blocks), 32)
    for i, b in enumerate(blocks):
        x[:, 32 * b:32 * b + 32] = torch.from_numpy(a[:, i]).to(DEV, torch.bfloat16)
    z = R.razer_gemm_mx_online(x, cw, sw, torch.float32)
    assert torch.equal(z.double().cpu(), torch.from_numpy(a.reshape(M, -1) @ w.T))
    assert R.razer_get_device_status() == 0


def test_a_group_of_2_31_rows():
    # more rows than 2^31 less a unit of the product: codes of 34 GB, checked at both ends and between
    T, N, K = (1 << 31) - 1, 2, 32
    if torch.cuda.mem_get_info()[0] < 72 << 30:
        pytest.skip("needs 72 GB of device memory")
    off = [5, T - 1]
    o = torch.tensor(off, dtype=torch.int32, device=DEV)
    ca, sa = bytes_of((T, K // 2), 0, 256, 1), bytes_of(R.razer_scale_tiles_shape(T, K, groups=1), 120, 135, 2)
    sa[:, 0].view(-1, 32, 4, 4)[..., 1:] = 0  # what lies past K / 32 = 1 scale
    c, s = ref.random_packed(N, K, "mxfp4", 3)
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device=DEV)
    R.razer_gemm_mx_grouped(ca, sa, o, dev(c)[None], dev(ref.tile(s))[None], out=y)
    assert R.razer_get_device_status() == 0
    rows = np.unique(np.concatenate([np.arange(off[0], 400), np.arange(T - 400, off[1]), (1 << 30) + np.arange(-200, 200),
                                     np.random.default_rng(0).integers(off[0], off[1], 400)]))
    at = torch.from_numpy(rows).to(DEV)
    i = at - off[0]
    scales = sa[i // 128, 0, (i % 32) * 16 + i % 128 // 32 * 4]
    a = ref.values(ca[at].cpu().numpy(), scales.cpu().numpy()[:, None], "mxfp4")
    r, _, bound = ref.product(a, ref.values(c, s, "mxfp4"))
    ref.check(y[at], r, bound)
    assert (y[:5] == 7).all() and (y[T - 1] == 7).all()


def test_falling_offsets_of_many_groups():
    # 32768 "groups" of every row: 2^31 units of the product, were they taken as they are.  Nothing
    # outside the output is written, the work is that of the sizes, and the call is reported
    T, N, K, E = 1 << 17, 4096, 32, 1 << 16
    o = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    o[1::2] = T
    cw, sw = bytes_of((E, N, K // 2), 0, 256, 1), bytes_of((E, N // 128, 1, 512), 120, 135, 2)
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(3)).to(DEV, torch.bfloat16)
    guard = 1 << 20
    room = torch.full((2 * guard + T * N,), 7.0, dtype=torch.bfloat16, device=DEV)
    y = room[guard:-guard].view(T, N)
    codes, tiles = R.razer_quantize_mx(x, o)
    assert R.razer_get_device_status() == 1
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for call in (lambda: R.razer_gemm_mx_grouped(codes, tiles, o, cw, sw, out=y), lambda: R.razer_gemm_mx_grouped_online(x, o, cw, sw, out=y)):
        start.record()
        call()
        end.record()
        assert R.razer_get_device_status() == 1
        assert start.elapsed_time(end) < 2000.0  # 2.2 million units; all of them would take tens of seconds
        assert (room[:guard] == 7).all() and (room[-guard:] == 7).all()
