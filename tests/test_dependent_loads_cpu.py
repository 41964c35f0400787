"""Kernels that start while the kernel before them still writes (programmatic
dependents, csrc/pdl.cuh) read what it wrote after their wait.  The read-only
path is for data that is constant while the kernel runs, and the compiler may
move such a load before the wait; so these kernels use neither __ldg nor const
__restrict__ parameters.  Checked on the sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_flashattention_gb300", "csrc")


def code(name):
    s = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", s, flags=re.S)


DEPENDENT = sorted(f for f in os.listdir(CSRC) if f != "pdl.cuh" and '#include "pdl.cuh"' in code(f))


def read_only(text):
    return re.findall(r"__ldg\s*\(|const\s+\w+\s*\*\s*__restrict__|ld\.global\.nc", text)


def test_the_files_are_found():
    assert {"batch.cu", "decode_fp4.cu", "kv_fp4.cu"} <= set(DEPENDENT)


@pytest.mark.parametrize("name", DEPENDENT)
def test_no_read_only_loads(name):
    assert not read_only(code(name))


def test_combine_of_the_split_decode():
    """decode.cu launches its combine as a dependent of the split kernel."""
    kernels = re.split(r"(?=__global__)", code("decode.cu"))
    dependent = [k for k in kernels if "griddepcontrol.wait" in k]
    assert len(dependent) == 1 and "lse_combine_kernel" in dependent[0]
    body = dependent[0][:dependent[0].index("launch_decode_t")]
    assert not read_only(body)
