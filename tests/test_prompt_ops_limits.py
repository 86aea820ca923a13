"""Limits of the prompt operators that hold on the host (no GPU needed)."""
import ctypes
import os
import re
import subprocess
import sys

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


# ---- errors of the runtime --------------------------------------------------------------------------
def test_a_missing_device_is_an_error_of_the_runtime():
    """In a process of its own that sees no device, so that nothing can be launched."""
    code = """
import sys
sys.path.insert(0, sys.argv[1])
from persistent_tile_pipelined_b200 import tre
P = 1 << 20
a = tre.tre_attention(8, 2, 128, 0, 5, 9, 8 * 128, 128, 128, 9 * 128, 128, 9 * 128, 8 * 128, 128, 0.1)
status = [tre.tre_prompt_attention(a, P, P, P, 0, 0, P),
          tre.tre_mxfp4_matmul(P, 64, P, 0, 1, 5, 9, 64, tre.TRE_F32, P, 9),
          tre.tre_mxfp4_quantize(P, tre.TRE_F32, 4, 64, 64, P),
          tre.tre_mxfp4_dequantize(P, 4, 64, tre.TRE_F32, P),
          tre.tre_add_rmsnorm(P, 64, 0, 0, 0, P, 1e-5, 5, 64, P, 64, P, 64)]
assert status == [tre.TRE_ERR_CUDA] * 5, status
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", code, root], capture_output=True, text=True,
                         env=dict(os.environ, CUDA_VISIBLE_DEVICES=""), timeout=120)
    assert run.returncode == 0, run.stderr[-2000:]


# ---- the end of a CTA ---------------------------------------------------------------------------
@pytest.mark.parametrize("source", ["prompt_attention.cu", "mxfp4_matmul.cu"])
def test_copies_and_products_end_before_the_cta_whoever_gave_up(source):
    """The threads that issue copies and products wait for the last of them in every path: one
    that has finished its loop cannot know that another role gives up later, after which the
    shared and tensor memory go to another CTA.  (Read, not run: a wait that runs out beside
    work in flight would be a fault on purpose.)"""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, source)).read())
    calls = [m.start() for m in re.finditer(r"tc::settle(_copies)?\(", text)]
    assert len(calls) >= 2
    for at in calls:
        before = text[:at].rstrip()
        assert before.endswith((";", "}")) or before.endswith("if (first_job < jobs)"), before[-80:]
    assert "tc::settle_copies(" in text and re.search(r"tc::settle\(", text)
    # whole loops over the barriers of their own are not left beside them
    assert "mbar_try_wait(" not in text


# ---- waits that run out ---------------------------------------------------------------------------
@pytest.mark.parametrize("clocks", [-1, 4_000_000_001, 1 << 62])
def test_a_wait_to_run_out_stays_short(clocks):
    assert tre.tre_debug_ops_timeout(clocks) == tre.TRE_ERR_INVALID_ARG


# ---- arguments of the torch forms -----------------------------------------------------------------
def test_a_tensor_without_dimensions_is_refused_like_every_other():
    torch = pytest.importorskip("torch")
    from persistent_tile_pipelined_b200 import ops
    for call in (lambda t: ops.mxfp4_dequantize(t.byte(), 32), ops.mxfp4_quantize):
        with pytest.raises(ValueError, match="dimensions|row"):
            call(torch.tensor(1.0))
