"""Limits of the prompt operators that hold on the host (no GPU needed)."""
import ctypes

import pytest

from persistent_tile_pipelined_b200 import build

build.build_engine()
from persistent_tile_pipelined_b200 import tre  # noqa: E402


# ---- attention: the scale -----------------------------------------------------------------------
@pytest.mark.parametrize("scale,status", [
    (1e-45, tre.TRE_OK), (1.0, tre.TRE_OK), (2.3e38, tre.TRE_OK),
    (2.4e38, tre.TRE_ERR_INVALID_ARG), (2.99e38, tre.TRE_ERR_INVALID_ARG)])
def test_attention_scale_is_finite_in_base_2(scale, status):
    """The kernel multiplies by scale log2(e), which has to be a number."""
    a = tre.tre_attention(8, 2, 128, 0, 5, 9, 8 * 128, 128, 128, 9 * 128, 128, 9 * 128, 8 * 128,
                          128, scale)
    b = ctypes.c_size_t()
    assert tre.lib.tre_prompt_attention_workspace(ctypes.byref(a), 148, ctypes.byref(b)) == status
