"""What the sources of the microscaled kernels have to keep to, checked on the
CPU: rules whose breach a GPU test could only show by hanging or faulting."""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantization_razer_b200", "csrc")


def kernels(name):
    """{kernel name: body} of a source file, comments left out."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    found = {}
    for m in re.finditer(r"__global__\s+void\s+__launch_bounds__\([^)]*\)\s+(\w+)\(", text):
        at = text.index("{", text.index(")\n{", m.end()))
        depth = 0
        for end in range(at, len(text)):
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            if depth == 0:
                break
        found[m.group(1)] = text[at:end]
    return found


@pytest.mark.parametrize("name", ["mx_gemm.cu", "gemm.cu"])
def test_dependents_are_let_in_after_tensor_memory_is_allocated(name):
    # A dependent grid that is resident before this one has its tensor memory
    # may take the columns and then wait for this grid: neither would end.
    allocating = {k: b for k, b in kernels(name).items() if "tcgen05.alloc" in b}
    assert allocating
    for kernel, body in allocating.items():
        triggers = [m.start() for m in re.finditer(r"pdl_trigger\(\)|launch_dependents", body)]
        if not triggers:
            continue  # dependents start when the grid has ended
        alloc = body.index("tcgen05.alloc")
        assert len(triggers) == 1, kernel  # one warp's: any thread's trigger counts for its block
        assert triggers[0] > alloc, kernel
        between = body[alloc:triggers[0]]
        assert "}" not in between and "else" not in between, kernel  # the warp that allocates


def test_tables_of_host_threads(tmp_path):
    # what a first call finds out is published whole: the thread sanitizer over the table the products keep it in
    here, exe = os.path.dirname(os.path.abspath(__file__)), str(tmp_path / "per_device_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=thread", "-pthread", "-I", CSRC, os.path.join(here, "per_device_check.cpp"), "-o", exe],
                   check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    if "FATAL: ThreadSanitizer" in out.stderr:
        pytest.skip("the thread sanitizer cannot map its memory here")
    assert out.returncode == 0 and "all checks passed" in out.stdout, out.stdout + out.stderr
    with open(os.path.join(CSRC, "mx_gemm.cu")) as f:
        assert not re.search(r"static (bool|int) \w+\[", f.read())  # no table of plain values beside it
