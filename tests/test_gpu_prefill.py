"""The prompt path of an engine (Engine.prefill, Engine.prefill_layers) against the fp64
oracle's decode steps token by token: same caches, same hidden states, and decode steps that
continue from either.  Bar: the framework's own 2e-2 (normwise); the path's activations are
bf16 where the decode step's are fp32, an error of a few times 2^-8."""
import numpy as np
import pytest

import oracle
from persistent_tile_pipelined_b200.synth import bf16_to_f32, token_id
from persistent_tile_pipelined_b200.synth import workloads as W

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from persistent_tile_pipelined_b200 import ops, tre  # noqa: E402

TOL = 2e-2
ORC = oracle.Oracle(64)


def relerr(g, o):
    g, o = np.asarray(g, np.float64), np.asarray(o, np.float64)
    return float(np.abs(g - o).max() / max(np.abs(o).max(), 1e-30))


def cache_words(t):
    return bf16_to_f32(t.view(torch.int16).cpu().numpy().view(np.uint16))


@pytest.mark.parametrize("wl,pieces", [
    (W.TINY.replace(prefill=0, decode_steps=80), [70]),
    (W.TINY.replace(prefill=33, decode_steps=60), [1, 40, 9]),
    (W.TINY.replace(prefill=5, decode_steps=50, n_q_heads=8, n_kv_heads=1, head_dim=128), [40]),
], ids=["empty-cache", "pieces", "mqa-128"])
def test_prefill_then_decode(wl, pieces):
    model = W.gen_gqa_model(wl)
    dev = tre.upload_gqa_model(model)
    eng = tre.Engine(tre.config_from_workload(wl), dev)
    toks = [token_id(wl.seed, wl.vocab, i) for i in range(sum(pieces) + 1)]
    want_h = []
    for i, t in enumerate(toks):
        ref_logits, hid = ORC.decode_step(wl, model, t, wl.prefill + i)
        want_h.append(hid[-1])
    at = 0
    for n in pieces:
        x_out = torch.empty((n, wl.hidden), device="cuda")
        ids = toks[at:at + n]
        eng.prefill(ids if at else torch.tensor(ids, dtype=torch.int32, device="cuda"),
                    wl.prefill + at, x_out=x_out)
        assert relerr(x_out.cpu().numpy(), want_h[at:at + n]) <= TOL
        at += n
    end = wl.prefill + at
    for l in range(wl.n_layers):
        for name in ("k_cache", "v_cache"):
            got, want = cache_words(dev[name][l]), bf16_to_f32(model[name][l])
            assert relerr(got[:, :end], want[:, :end]) <= TOL
            assert (got[:, end:] == 0).all()
    logits = torch.empty(wl.vocab, device="cuda")
    eng.step(toks[-1], end, logits)
    torch.cuda.synchronize()
    assert eng.status() == (0, 0) and tre.tre_ops_status() == 0
    assert relerr(logits.cpu().numpy(), ref_logits) <= TOL
    eng.close()


def test_prefill_without_output_fills_the_same_caches():
    wl = W.TINY.replace(prefill=0, decode_steps=140)
    model = W.gen_gqa_model(wl)
    toks = [token_id(wl.seed, wl.vocab, i) for i in range(130)]
    got = []
    for want_output in (False, True):
        dev = tre.upload_gqa_model(model)
        eng = tre.Engine(tre.config_from_workload(wl), dev)
        x_out = torch.empty((130, wl.hidden), device="cuda") if want_output else None
        eng.prefill(toks, 0, x_out=x_out)
        got.append([t.clone() for t in dev["k_cache"] + dev["v_cache"]])
        eng.close()
    assert all(torch.equal(a, b) for a, b in zip(*got))


MOE = W.MOE4.replace(name="moe-prefill", n_layers=1, hidden=512, n_q_heads=8, n_kv_heads=2,
                     head_dim=64, prefill=21, decode_steps=30, n_experts=12, top_k=3, n_shared=1,
                     expert_ffn=192, seed=77, weight_format="fp4")


@pytest.mark.parametrize("n_shared", [1, 2])
def test_prefill_layers_of_fp4_experts(n_shared):
    """One layer (with several, a token whose routing is a near tie would move the later
    layers): every token whose selection boundary is wider than the bf16 path's noise in
    the scores (3 * 2^-8 of a score below 1) must match the oracle."""
    wl = MOE.replace(n_shared=n_shared)
    model = W.gen_moe_model(wl, with_experts=True)
    ex = model["experts"]
    dev = tre.upload_moe_model(wl, model, expert_fn=lambda l, e: ex[l][e])
    eng = tre.Engine(tre.config_from_workload(wl), dev)
    T = 25
    rng = np.random.default_rng(3)
    xs = rng.standard_normal((T, wl.hidden)).astype(np.float32)
    want, clear = [], []
    for t in range(T):
        y, _, _, scores = ORC.moe_layer_step(
            wl, model["layers"][0], model["k_cache"][0], model["v_cache"][0],
            lambda e: ex[0][e], wl.prefill + t, xs[t], want_scores=True)
        s = np.sort(np.asarray(scores, np.float64))[::-1]
        want.append(y)
        clear.append(s[wl.top_k - 1] - s[wl.top_k] > 3 * 2.0 ** -8)
    clear = np.array(clear)
    assert clear.sum() >= 5
    x_in = torch.from_numpy(xs).cuda()
    out = eng.prefill_layers(x_in, wl.prefill)
    assert torch.equal(x_in.cpu(), torch.from_numpy(xs))
    got = out.cpu().numpy()
    assert np.isfinite(got).all()
    assert relerr(got[clear], np.array(want)[clear]) <= TOL
    # a decode step goes on from the caches
    y = torch.empty(wl.hidden, device="cuda")
    x = torch.from_numpy(rng.standard_normal(wl.hidden).astype(np.float32)).cuda()
    eng.layers_step(x, y, wl.prefill + T)
    ref, idx, _ = ORC.moe_layer_step(wl, model["layers"][0], model["k_cache"][0],
                                     model["v_cache"][0], lambda e: ex[0][e], wl.prefill + T,
                                     x.cpu().numpy())
    torch.cuda.synchronize()
    assert eng.status() == (0, 0) and tre.tre_ops_status() == 0
    assert relerr(y.cpu().numpy(), ref) <= TOL
    eng.close()


def test_upload_quantises_bf16_experts():
    wl = MOE
    plain = wl.replace(weight_format="bf16")
    model = W.gen_moe_model(wl)
    dev = tre.upload_moe_model(wl, model, expert_fn=lambda l, e: W.gen_expert(plain, l, e))
    gate = dev["layers"][0][10]
    words = np.stack([W.gen_expert(plain, 0, e)[0] for e in range(wl.n_experts)])
    w = torch.from_numpy(words.view(np.int16)).view(torch.bfloat16).cuda()
    assert torch.equal(gate, ops.mxfp4_quantize(w))
    down = dev["layers"][0][12]
    words = np.stack([W.gen_expert(plain, 0, e)[2] for e in range(wl.n_experts)])
    w = torch.from_numpy(words.view(np.int16)).view(torch.bfloat16).cuda()
    assert torch.equal(down, ops.mxfp4_quantize(w))


def test_prefill_refuses():
    wl = W.TINY
    dev = tre.upload_gqa_model(W.gen_gqa_model(wl))
    eng = tre.Engine(tre.config_from_workload(wl), dev)
    cap = wl.kv_capacity
    for tokens, pos, status in [([1] * 10, cap - 9, tre.TRE_ERR_POS_RANGE),
                                ([1], -1, tre.TRE_ERR_POS_RANGE),
                                ([wl.vocab], 0, tre.TRE_ERR_INVALID_ARG),
                                ([-1], 0, tre.TRE_ERR_INVALID_ARG),
                                (torch.zeros(2, 2, dtype=torch.int32), 0, tre.TRE_ERR_INVALID_ARG),
                                (torch.zeros(2), 0, tre.TRE_ERR_INVALID_ARG)]:
        with pytest.raises(tre.TreError) as e:
            eng.prefill(tokens, pos)
        assert e.value.status == status
    eng.prefill([], 0)
    with pytest.raises(tre.TreError):
        eng.prefill([1, 2], 0, x_out=torch.empty(3, wl.hidden, device="cuda"))
    with pytest.raises(tre.TreError):
        eng.prefill_layers(torch.zeros(2, wl.hidden - 1, device="cuda"))
    eng.close()
    fp8 = wl.replace(weight_format="fp8")
    eng = tre.Engine(tre.config_from_workload(fp8), tre.upload_gqa_model(W.gen_gqa_model(fp8)))
    with pytest.raises(tre.TreError) as e:
        eng.prefill([1], 0)
    assert e.value.status == tre.TRE_ERR_UNSUPPORTED
    eng.close()
