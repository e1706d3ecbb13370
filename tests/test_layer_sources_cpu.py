"""Orders of steps in the kernels' sources that no run can be made to show safely."""

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_precision_x32_gb300", "csrc")


def kernels():
    """(name, body) of every __global__ function."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for part in text.split("__global__")[1:]:
            at = part.index("{")
            depth = 0
            for i in range(at, len(part)):
                depth += {"{": 1, "}": -1}.get(part[i], 0)
                if depth == 0:
                    yield re.findall(r"(\w+)\s*\(", part[:at])[1], part[at:i + 1]
                    break


def test_the_next_kernel_starts_only_once_tensor_memory_is_held():
    """A block of the next kernel that took tensor memory first would wait for this kernel's end, and this kernel for the
    columns: let_next_start() comes behind a barrier that follows the allocation."""
    found = 0
    for name, body in kernels():
        if "tmem_alloc" in body and "let_next_start" in body:
            found += 1
            steps = [body.index(s) for s in ("tmem_alloc", "__syncthreads", "let_next_start")]
            assert steps == sorted(steps), name
    assert found


def test_an_overlapped_kernel_waits_for_the_stream():
    """Every kernel that lets the next one start waits for those in front of it, ahead of its first use of memory."""
    overlapped = [(n, b) for n, b in kernels() if "let_next_start" in b]
    assert len(overlapped) >= 10
    for name, body in overlapped:
        assert "wait_for_stream" in body, name
