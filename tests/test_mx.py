"""Host side of the microscaled 4-bit calls: layouts, sizes, and every refusal
before a launch (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import bit_quantization_razer_b200 as R
from bit_quantization_razer_b200.build import build
from tests import mx_reference as ref

FAKE = ctypes.c_void_p(0x1000)  # 16-byte aligned; never dereferenced (validation fails first)
ODD = ctypes.c_void_p(0x1004)
BYTE = ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module")
def lib():
    build()
    return R.load()


def test_reference_quantizer_against_every_grid_point_and_midpoint():
    grid = ref.E2M1[:8]
    pts = np.concatenate([grid, (grid[:-1] + grid[1:]) / 2, np.nextafter((grid[:-1] + grid[1:]) / 2, 9), [6.5, 7.9]])
    x = np.zeros((len(pts), 32))
    x[:, 0], x[:, 1] = pts, 4.0  # the 4 makes the scale 1
    codes, scales = ref.quantize(x)
    for i, p in enumerate(pts):
        top = max(p, 4.0)
        e = int(np.floor(np.log2(top))) - 2
        assert scales[i, 0] == e + 127
        d = np.abs(grid - p / 2.0 ** e)
        best = np.flatnonzero(d == d.min())
        want = best[0] if len(best) == 1 else next(b for b in best if b % 2 == 0)
        assert codes[i, 0] == want, p


def test_tile_layout_round_trip():
    rng = np.random.default_rng(0)
    rows = rng.integers(0, 256, (300, 11)).astype(np.uint8)
    assert np.array_equal(ref.untile(ref.tile(rows), 300, 11), rows)
    off = [5, 5, 140, 141, 269, 290]
    got = ref.untile(ref.tile(rows, off), 300, 11, off)
    assert np.array_equal(got[5:290], rows[5:290])
    # groups never share a tile row, and T / 128 + E tile rows hold them all
    rng = np.random.default_rng(1)
    for _ in range(300):
        E, T = int(rng.integers(1, 12)), int(rng.integers(1, 2000))
        off = np.sort(rng.integers(0, T + 1, E + 1))
        tr, at = ref.slots(T, off)
        used = tr[tr >= 0] * 128 + at[tr >= 0]
        assert len(set(used)) == len(used)
        owner = {}
        for e in range(E):
            for t in set(tr[off[e]:off[e + 1]]):
                assert owner.setdefault(t, e) == e
        assert tr.max(initial=-1) < T // 128 + E


def test_sizes(lib):
    assert lib.razer_scale_tiles_size(5, 300, 160, 0) == 3 * 2 * 512
    assert lib.razer_scale_tiles_size(2, 300, 160, 0) == 3 * 3 * 512
    assert lib.razer_scale_tiles_size(5, 300, 160, 7) == (2 + 7) * 2 * 512
    assert lib.razer_scale_tiles_size(5, 0, 160, 0) == 0
    assert lib.razer_scale_tiles_size(0, 300, 160, 0) == 0  # RaZeR weights have no tiles
    assert R.razer_scale_tiles_shape(300, 160, "nvfp4") == (3, 3, 512)
    assert R.razer_scale_tiles_shape(300, 160, "mxfp4", 7) == (9, 2, 512)
    assert R.razer_workspace_size(R.RAZER_OP_GEMM_MX_ONLINE, 300, 64, 160) == 24064 + 3 * 2 * 512
    assert R.razer_gemm_mx_grouped_workspace_size(300, 160, 7) == 24064 + 9 * 2 * 512  # 43 rows a group
    assert R.razer_gemm_mx_grouped_workspace_size(0, 160, 7) == 0
    # few rows are quantized inside the product
    assert R.razer_workspace_size(R.RAZER_OP_GEMM_MX_ONLINE, 16, 64, 160) == 0 < R.razer_workspace_size(R.RAZER_OP_GEMM_MX_ONLINE, 17, 64, 160)
    assert R.razer_gemm_mx_grouped_workspace_size(7 * 4, 160, 7) == 0 < R.razer_gemm_mx_grouped_workspace_size(7 * 4 + 1, 160, 7)


def test_quantizer_refusals(lib):
    q = lib.razer_quantize_mx
    a = lambda x=FAKE, dt=1, M=4, K=64, off=None, E=0, c=FAKE, s=FAKE: q(x, dt, M, K, off, E, c, s, None)
    assert a(K=48) == 2 and a(K=16) == 2 and a(M=-1) == 2 and a(K=-32) == 2 and a(M=1 << 31) == 2
    assert a(dt=2) == 4 and a(dt=9) == 1
    assert a(x=None) == 1 and a(c=None) == 1 and a(s=None) == 1
    assert a(x=ODD) == 3 and a(c=ODD) == 3 and a(s=ODD) == 3
    assert a(E=2) == 1 and a(E=-1, off=FAKE) == 2 and a(E=2, off=BYTE) == 3
    assert a(M=0, x=None) == 0 and a(K=0, x=None) == 0  # empty: nothing is done
    d = lib.razer_dequant_mx
    b = lambda c=FAKE, s=FAKE, M=4, K=64, off=None, E=0, o=FAKE, dt=2: d(c, s, M, K, off, E, o, dt, None)
    assert b(K=48) == 2 and b(M=-1) == 2 and b(dt=7) == 1 and b(c=None) == 1 and b(s=None) == 1 and b(o=None) == 1
    assert b(c=ODD) == 3 and b(s=ODD) == 3 and b(o=ODD) == 3 and b(E=1) == 1
    assert b(M=0, c=None) == 0
    t = lib.razer_tile_scales
    c = lambda s=FAKE, B=1, R_=4, C=4, off=None, E=0, o=FAKE: t(s, B, R_, C, off, E, o, None)
    assert c(B=-1) == 2 and c(R_=-1) == 2 and c(C=-1) == 2 and c(E=-1) == 2
    assert c(B=2, E=3, off=FAKE) == 2      # groups go with one matrix
    assert c(E=3) == 1 and c(E=3, off=BYTE) == 3
    assert c(s=None) == 1 and c(o=None) == 1 and c(o=ODD) == 3
    assert c(B=1 << 20, R_=1 << 20, C=1 << 20) == 2
    assert c(B=0, s=None) == 0 and c(R_=0, s=None) == 0


def test_product_refusals(lib):
    g = lib.razer_gemm_mx
    def a(ca=FAKE, sa=FAKE, ta=None, M=4, cw=FAKE, sw=FAKE, tw=None, fmt=5, N=8, K=64, act=0, y=FAKE, dt=1):
        return g(ca, sa, ta, M, cw, sw, tw, fmt, N, K, act, y, dt, None)
    for fmt in (0, 1):
        assert a(fmt=fmt) == 6            # the remapped code has no tensor-core form
    for fmt in (3, 4, 9, -1):
        assert a(fmt=fmt) == 1
    assert a(K=48) == 2 and a(M=-1) == 2 and a(N=-1) == 2 and a(N=1 << 31) == 2 and a(K=1 << 31) == 2
    assert a(act=1, N=9) == 2 and a(act=2) == 1
    assert a(dt=5) == 1
    assert a(ca=None) == 1 and a(sa=None) == 1 and a(cw=None) == 1 and a(sw=None) == 1 and a(y=None) == 1
    assert a(fmt=2) == 1 and a(fmt=2, ta=FAKE) == 1 and a(fmt=2, tw=FAKE) == 1   # NVFP4 needs both tensor scales
    for k in ("ca", "sa", "cw", "sw", "y"):
        assert a(**{k: ODD}) == 3, k
    assert a(ta=BYTE) == 3 and a(tw=BYTE) == 3
    assert a(M=0, ca=None, sa=None, y=None) == 0 and a(N=0, cw=None, sw=None, y=None) == 0
    h = lib.razer_gemm_mx_grouped
    def b(off=FAKE, E=2, T=4, N=8, K=64, fmt=5, tw=None, ta=None):
        return h(FAKE, FAKE, ta, T, off, E, FAKE, FAKE, tw, fmt, N, K, 0, FAKE, 1, None)
    assert b(E=0) == 2 and b(E=-1) == 2 and b(off=None) == 1 and b(off=BYTE) == 3
    assert b(E=1 << 20, N=1 << 12) == 2   # E * N beyond the row index
    assert b(T=0) == 0 and b(N=0) == 0


def test_online_refusals(lib):
    g = lib.razer_gemm_mx_online
    def a(x=FAKE, xdt=1, M=40, cw=FAKE, sw=FAKE, N=8, K=64, act=0, y=FAKE, dt=1, ws=FAKE, wsb=1 << 20):
        return g(x, xdt, M, cw, sw, N, K, act, y, dt, ws, wsb, None)
    need = R.razer_workspace_size(R.RAZER_OP_GEMM_MX_ONLINE, 40, 8, 64)
    assert a(xdt=2) == 4 and a(xdt=8) == 1 and a(K=48) == 2 and a(x=None) == 1 and a(x=ODD) == 3
    assert a(ws=None) == 5 and a(wsb=need - 1) == 5 and a(ws=ODD) == 3
    assert a(act=1, N=9) == 2 and a(act=7) == 1 and a(cw=None) == 1 and a(sw=ODD) == 3
    assert a(M=0, x=None, ws=None, wsb=0) == 0
    h = lib.razer_gemm_mx_grouped_online
    def b(off=FAKE, E=2, T=40, ws=FAKE, wsb=1 << 20):
        return h(FAKE, 1, T, off, E, FAKE, FAKE, 8, 64, 0, FAKE, 1, ws, wsb, None)
    assert b(E=0) == 2 and b(off=None) == 1 and b(off=BYTE) == 3 and b(ws=None) == 5
    assert b(wsb=R.razer_gemm_mx_grouped_workspace_size(40, 64, 2) - 1) == 5


def test_older_calls_refuse_mxfp4(lib):
    f = 5
    assert lib.razer_quantize_weights(FAKE, 0, 4, 32, FAKE, FAKE, FAKE, f, None) == 1
    assert lib.razer_quantize_acts(FAKE, 1, 4, 32, None, FAKE, FAKE, FAKE, None, f, None) == 1
    assert lib.razer_dequant(FAKE, FAKE, FAKE, f, 4, 32, FAKE, 2, None) == 1
    assert lib.razer_gemv(FAKE, 0, 1, FAKE, FAKE, FAKE, f, 64, 128, FAKE, 2, FAKE, 1 << 20, None) == 1
    assert lib.razer_gemm(FAKE, 1, 64, FAKE, FAKE, FAKE, f, 64, 128, FAKE, 1, FAKE, 1 << 20, None) == 1
    assert lib.razer_gemm_w4a4(FAKE, FAKE, FAKE, f, 64, FAKE, FAKE, FAKE, 0, 64, 64, FAKE, 1, FAKE, 1 << 20, None) == 1
    V = (ctypes.c_float * 1)(5.0)
    assert lib.razer_quantize_variant(FAKE, 0, 4, 32, 32, f, V, 1, FAKE, FAKE, FAKE, None) == 1


def test_python_calls_refuse_what_the_library_cannot_see():
    # host tensors, other shapes, other types and strides: refused before any call
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    u8 = torch.zeros(4, 32, dtype=torch.uint8)
    t = torch.zeros(1, 1, 512, dtype=torch.uint8)
    for call in (lambda: R.razer_quantize_mx(x), lambda: R.razer_dequant_mx(u8, t), lambda: R.razer_tile_scales(u8),
                 lambda: R.razer_gemm_mx(u8, t, u8, t), lambda: R.razer_gemm_mx_online(x, u8, t),
                 lambda: R.razer_quantize_mx(x[0]), lambda: R.razer_gemm_mx_grouped(u8, t, None, u8, t),
                 lambda: R.razer_gemm_mx_grouped_online(x, None, u8, t), lambda: R.razer_tile_scales(u8.view(1, 4, 32), torch.zeros(2))):
        with pytest.raises(ValueError):
            call()


def test_plain_c_consumer(lib, tmp_path):
    # the header's microscaled calls from a C program, every warning an error
    import os
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    libdir, exe = os.path.join(root, "bit_quantization_razer_b200"), str(tmp_path / "mx_abi_consumer")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(root, "include"),
                    os.path.join(root, "tests", "mx_abi_consumer.c"), "-L", libdir, "-lrazer", "-Wl,-rpath," + libdir, "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stderr
    assert "all checks passed" in out.stdout
