"""The microscaled products where their values are far from 1: gates whose
exponential nears the end of fp32's range."""
import numpy as np
import pytest
import torch

import bit_quantization_razer_b200 as R
from tests import mx_reference as ref
from tests.gpu_helpers import cuda

pytestmark = [pytest.mark.gpu, cuda]
DEV = "cuda:0"


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


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
