"""The order of a kernel's set-up in the sources: CTAs of the next kernel of a
stream may start once every CTA of this one has called grid_dep_launch, and
may take tensor memory at once.  So a kernel calls it only behind the barrier
that follows its own allocation: otherwise a dependent could hold the columns that
this grid still waits for, and then wait for this grid."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "discrete_diffusion_moe_b200", "csrc")


def _kernels():
    """(file:kernel, body) of every __global__ function."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__", text):
            start = text.index("{", m.start())
            name = re.search(r"(\w+)\s*\(", re.sub(r"__launch_bounds__\([^{]*?\)\s*\n?\s*(?=\w)", "", text[m.end():start]))
            depth, at = 1, start + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
            yield f"{os.path.basename(path)}:{name.group(1) if name else m.start()}", text[start:at]


KERNELS = dict(_kernels())
WITH_TMEM = sorted(k for k, body in KERNELS.items() if re.search(r"\btmem_alloc(_pair)?\(", body))


def test_the_kernels_with_tensor_memory_are_found():
    files = {k.split(":")[0] for k in WITH_TMEM}
    assert files == {"attention_tc.cuh", "gemm_tc.cuh", "gemm_pair.cuh", "moe_pair.cuh", "fp8_gemm.cuh", "fp8_stream.cuh"}


@pytest.mark.parametrize("kernel", WITH_TMEM)
def test_dependents_start_after_the_tensor_memory_is_held(kernel):
    body = KERNELS[kernel]
    alloc = re.search(r"\btmem_alloc(_pair)?\(", body).start()
    held = body.index("__syncthreads()", alloc)
    launches = [m.start() for m in re.finditer(r"\bgrid_dep_launch\(\)", body)]
    assert len(launches) == 1 and launches[0] > held
    assert body.index("grid_dep_wait()") < launches[0]
