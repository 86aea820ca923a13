"""A wait of the prompt operators that runs out of time: the kernel ends, the status word says
so, and the context stays usable."""
import time

import pytest

from persistent_tile_pipelined_b200.synth import workloads as W

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from persistent_tile_pipelined_b200 import ops, tre  # noqa: E402


@pytest.fixture(autouse=True)
def _clean():
    assert tre.tre_ops_status() == 0
    yield
    assert tre.tre_ops_status() == 0


def run_out(clocks=20_000_000):  # 10 ms
    assert tre.tre_debug_ops_timeout(clocks, torch.cuda.current_stream().cuda_stream) == tre.TRE_OK


@pytest.mark.parametrize("clocks", [0, 20_000_000])
def test_a_wait_gives_up_and_says_so(clocks):
    torch.cuda.synchronize()
    start = time.monotonic()
    run_out(clocks)
    assert tre.tre_ops_status() == tre.TRE_ERR_DEP_TIMEOUT
    took = time.monotonic() - start
    assert clocks / 2.5e9 <= took < 1.0  # at its limit, not at the operators' two seconds
    assert tre.tre_ops_status() == 0  # reading clears it


def test_operators_run_after_it():
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((5, 4, 64), generator=g, device="cuda").bfloat16()
    kv = torch.randn((2, 9, 64), generator=g, device="cuda").bfloat16()
    want = ops.prompt_attention(q, kv, kv)
    run_out()
    assert torch.equal(ops.prompt_attention(q, kv, kv), want)
    assert tre.tre_ops_status() == tre.TRE_ERR_DEP_TIMEOUT


def test_an_engine_reports_its_prompts_timeouts():
    wl = W.TINY
    eng = tre.Engine(tre.config_from_workload(wl), tre.upload_gqa_model(W.gen_gqa_model(wl)))
    run_out()
    assert eng.status() == (0, 0)  # no prompt of this engine: left for whom it concerns
    assert tre.tre_ops_status() == tre.TRE_ERR_DEP_TIMEOUT
    eng.prefill([1, 2, 3], 0)
    assert eng.status() == (0, 0)
    run_out()
    assert eng.status() == (tre.TRE_ERR_DEP_TIMEOUT, -1)
    assert eng.status() == (tre.TRE_ERR_DEP_TIMEOUT, -1)  # until it is reset
    eng.reset()
    assert eng.status() == (0, 0)
    eng.close()
