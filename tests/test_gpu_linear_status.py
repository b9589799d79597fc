"""csa_linear_q8_status takes away what it has seen and nothing else: a bit that a call on another stream raises between the
look and the clearing is the next look's.  The bounds-checked build's hook CSA_TEST_RAISE_BEFORE_CLEARING raises one
there, CSA_TEST_SHORT_EXTENTS the first (see test_gpu_serving_extents)."""
import os

import pytest
import torch

import deepseek_v4_compressed_wkv_gb300 as csa
from test_gpu_layer_bounds import run_on_the_bounds_checked_build
from test_gpu_linear_q8 import inputs

pytestmark = pytest.mark.gpu
BOUNDS = os.environ.get("CSA_LIBRARY_VARIANT") == "bounds"


@pytest.mark.skipif(not BOUNDS, reason="the hooks exist only in the bounds-checked build")
def test_a_bit_raised_meanwhile_is_left_to_the_next_look(monkeypatch):
    v = inputs(5, 200, 512)
    want = csa.linear_q8(*v)
    csa.linear_q8_status()
    monkeypatch.setenv("CSA_TEST_SHORT_EXTENTS", "rows")
    csa.linear_q8(*v)
    monkeypatch.delenv("CSA_TEST_SHORT_EXTENTS")
    monkeypatch.setenv("CSA_TEST_RAISE_BEFORE_CLEARING", "4")
    with pytest.raises(csa.CSAError, match="out of bounds"):
        csa.linear_q8_status()
    monkeypatch.delenv("CSA_TEST_RAISE_BEFORE_CLEARING")
    with pytest.raises(csa.CSAError, match="0x4: wait budget"):
        csa.linear_q8_status()
    csa.linear_q8_status()
    assert torch.equal(csa.linear_q8(*v), want)


if not BOUNDS:
    def test_on_the_bounds_checked_build():
        run_on_the_bounds_checked_build("test_gpu_linear_status.py")
