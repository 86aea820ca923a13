"""The prompt path at the full width of a layer of each stack, in pieces, against the engine's own
decode steps position by position (which the oracle's tests cover).  Bar: the framework's 2e-2
(normwise); the path's activations are bf16 where the decode step's are fp32."""
import pytest

from persistent_tile_pipelined_b200.synth import workloads as W

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from persistent_tile_pipelined_b200 import tre  # noqa: E402

TOL = 2e-2
GQA = W.LLAMA8B.replace(n_layers=1, vocab=0, prefill=64, decode_steps=330)
# all experts are chosen: a near tie between two would move a token
MOE = W.MOE4_FP4.replace(n_layers=1, n_experts=8, top_k=8, prefill=64, decode_steps=330)


def relerr(got, want):
    return float((got.double() - want.double()).abs().max() / want.double().abs().max())


@pytest.mark.parametrize("wl,upload", [
    (GQA, lambda wl: tre.upload_gqa_model(W.gen_gqa_model(wl))),
    (MOE, lambda wl: tre.upload_moe_model(wl, W.gen_moe_model(wl)))], ids=["gqa", "moe-fp4"])
@pytest.mark.parametrize("pieces", [[300], [1, 40, 259]], ids=str)
def test_prefill_like_decode_steps(wl, upload, pieces):
    dev = upload(wl)
    steps = dict(dev, k_cache=[c.clone() for c in dev["k_cache"]],
                 v_cache=[c.clone() for c in dev["v_cache"]])
    cfg = tre.config_from_workload(wl)
    T = sum(pieces)
    x = torch.randn((T, wl.hidden), generator=torch.Generator(device="cuda").manual_seed(7),
                    device="cuda")
    eng = tre.Engine(cfg, steps)
    want = torch.empty_like(x)
    for t in range(T):
        eng.layers_step(x[t], want[t], wl.prefill + t)
    assert eng.status() == (0, 0)
    eng.close()
    eng = tre.Engine(cfg, dev)
    at = 0
    for n in pieces:
        got = eng.prefill_layers(x[at:at + n], wl.prefill + at)
        assert relerr(got, want[at:at + n]) <= TOL
        at += n
    assert eng.status() == (0, 0)
    eng.close()
    end = wl.prefill + T
    for name in ("k_cache", "v_cache"):
        got, ref = (m[name][0].view(wl.n_kv_heads, wl.kv_capacity, wl.head_dim)
                    for m in (dev, steps))
        assert relerr(got[:, :end], ref[:, :end]) <= TOL
        assert torch.equal(got[:, end:], ref[:, end:])
