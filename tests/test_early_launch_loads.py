"""Kernels that are launched while their predecessor still runs (launch_early) read what that one may be
writing.  The non-coherent load path is specified for data that does not change during the kernel's life,
and the compiler may move such loads across the wait: the sources of these kernels must not use it.  No
GPU is needed: the sources are read."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deepseek_v4_compressed_wkv_gb300", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def early():
    return [f for f in sorted(os.listdir(CSRC)) if f.endswith(".cu") and "launch_early(" in code(f)]


def test_there_are_such_kernels():
    assert early() == ["attention.cu", "layer_ops.cu"]


@pytest.mark.parametrize("name", early())
def test_no_non_coherent_loads(name):
    text = code(name)
    # __restrict__ on a const pointer lets the compiler choose that path by itself
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in text, word


def test_the_wait_holds_back_the_loads_behind_it():
    text = code("tc_common.cuh")
    assert re.search(r'asm volatile\("griddepcontrol\.wait;" ::: "memory"\)', text)


@pytest.mark.parametrize("name", early())
def test_every_kernel_waits_before_it_touches_memory(name):
    """In each kernel the wait comes before the first use of a pointer that the launch was given."""
    bodies = re.split(r"__global__", code(name))[1:]
    assert bodies
    for body in bodies:
        at = body.index("griddep_wait();")
        assert not re.search(r"P\.(c\.)?(q|kv|out|lse|lens|page_table|first|mask|status|x|residual|gain|y|cache|in|record|part|part_ml|"
                             r"ticket|flag)\b\s*(\[|\+|->)", body[:at]), body[:200]
