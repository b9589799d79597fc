"""More refusals of the attention layer's operators that need no GPU."""
import ctypes

import pytest

import deepseek_v4_compressed_wkv_gb300 as csa


@pytest.mark.parametrize("scale", [3.4e38, 2.4e38])
def test_a_scale_that_overflows_in_base_2_is_refused(scale):
    """Scores are taken in base 2: scale * log2(e) has to be a number."""
    h = ctypes.c_void_p()
    assert csa.load_library().csa_attention_create(64, 512, 0, 0, scale, ctypes.byref(h)) == -1 and not h.value
    assert "scale" in csa.load_library().csa_last_error().decode()


def test_the_largest_scale_is_not_refused_for_itself():
    """2.35e38 * log2(e) is just below f32's end: what fails without a GPU is the device, not the scale."""
    h = ctypes.c_void_p()
    rc = csa.load_library().csa_attention_create(64, 512, 0, 0, 2.35e38, ctypes.byref(h))
    assert rc != -1
    csa.load_library().csa_attention_destroy(h)
