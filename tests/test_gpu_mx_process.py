"""The microscaled products as the first calls that a process makes: each test
runs in an interpreter of its own, where nothing has been set up yet."""
import os
import subprocess
import sys

import pytest

from tests.gpu_helpers import cuda

pytestmark = [pytest.mark.gpu, cuda]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEAD = """
import threading
import torch
import bit_quantization_razer_b200 as R
from bit_quantization_razer_b200.razer import load
load()
g = torch.Generator(device="cuda")
g.manual_seed(5)
def packed(rows, K, block=32):
    codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    fmt = "mxfp4" if block == 32 else "nvfp4"
    lo, hi = (125, 130) if block == 32 else (40, 80)
    return codes, torch.randint(lo, hi, R.razer_scale_tiles_shape(rows, K, fmt), dtype=torch.uint8, device="cuda", generator=g)
"""


def run(body):
    out = subprocess.run([sys.executable, "-c", HEAD + body], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.endswith("ok\n"), out.stdout + out.stderr


def test_first_calls_of_host_threads():
    # K is split over clusters by what the first call finds out: every thread's sums are joined in the same order
    run("""
cases = [(3, 200, 8192), (100, 512, 8192), (3, 200, 8192), (100, 512, 8192)]
args = [(packed(M, K), packed(N, K)) for M, N, K in cases]
torch.cuda.synchronize()
got, failed, gate = [[] for _ in cases], [], threading.Barrier(len(cases))
def calls(i):
    try:
        stream = torch.cuda.Stream()
        gate.wait()
        for _ in range(5):
            got[i].append(R.razer_gemm_mx(*args[i][0], *args[i][1], out_dtype=torch.float32, stream=stream))
        stream.synchronize()
    except Exception as e:
        failed.append(e)
threads = [threading.Thread(target=calls, args=(i,)) for i in range(len(cases))]
for t in threads: t.start()
for t in threads: t.join()
torch.cuda.synchronize()
assert not failed, failed
for i in range(len(cases)):
    want = R.razer_gemm_mx(*args[i][0], *args[i][1], out_dtype=torch.float32)
    assert len(got[i]) == 5 and all(torch.equal(y, want) for y in got[i]), i
assert R.razer_get_device_status() == 0
print("ok")
""")


@pytest.mark.parametrize("call", [
    "R.razer_gemm_mx(*packed(3, 4096), *packed(200, 4096), out=few)",
    "R.razer_gemm_mx(*packed(130, 96, 16), *packed(258, 96, 16), 'nvfp4', ts_a=one, ts_w=one, act='silu_mul', out=out)",
    "R.razer_gemm_mx_online(x, *packed(256, 96), out=y)",
])
def test_first_call_of_a_process_in_a_capture(call):
    # what a call does for the first time (attributes, occupancy, the driver's entry point) is not barred while capturing
    run("""
one = torch.ones(1, device="cuda")
x = torch.randn(100, 96, device="cuda", generator=g).bfloat16()
y = torch.zeros(100, 256, device="cuda", dtype=torch.bfloat16)
out = torch.zeros(130, 129, device="cuda", dtype=torch.float16)
operands = {}
real = packed
def packed(rows, K, block=32):  # made once, before the capture
    key = (rows, K, block)
    if key not in operands: operands[key] = real(rows, K, block)
    return operands[key]
CALL = lambda: %s
""" % call + """
few = torch.zeros(3, 200, device="cuda", dtype=torch.float32)
for args in ((3, 4096), (200, 4096), (130, 96, 16), (258, 96, 16), (256, 96)): packed(*args)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    result = CALL()
assert not result.any()  # captured, not run
graph.replay()
torch.cuda.synchronize()
captured = result.clone()
result.zero_()
assert captured.any() and torch.equal(CALL(), captured)
assert R.razer_get_device_status() == 0
print("ok")
""")
