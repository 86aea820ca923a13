"""The prompt path of an engine under an application's global settings."""
import contextlib

import numpy as np
import pytest

from persistent_tile_pipelined_b200.synth import token_id
from persistent_tile_pipelined_b200.synth import workloads as W

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from persistent_tile_pipelined_b200 import prefill, tre  # noqa: E402

MOE = W.MOE4.replace(name="moe-prefill", n_layers=1, hidden=512, n_q_heads=8, n_kv_heads=2,
                     head_dim=64, prefill=0, decode_steps=90, n_experts=12, top_k=3, n_shared=1,
                     expert_ffn=192, seed=77, weight_format="fp4")


@contextlib.contextmanager
def tf32():
    before = torch.get_float32_matmul_precision()
    torch.set_float32_matmul_precision("high")
    try:
        yield
    finally:
        torch.set_float32_matmul_precision(before)


SETTINGS = {"tf32": tf32, "autocast-bf16": lambda: torch.autocast("cuda", torch.bfloat16),
            "autocast-fp16": lambda: torch.autocast("cuda", torch.float16)}


@pytest.fixture(scope="module")
def stacks():
    """Engines of both kinds and what each gives for 80 positions without any setting."""
    gqa = W.TINY.replace(prefill=0, decode_steps=90)
    moe = MOE
    model = W.gen_moe_model(moe, with_experts=True)
    ex = model["experts"]
    engines = {"gqa": tre.Engine(tre.config_from_workload(gqa),
                                 tre.upload_gqa_model(W.gen_gqa_model(gqa))),
               "moe": tre.Engine(tre.config_from_workload(moe), tre.upload_moe_model(
                   moe, model, expert_fn=lambda l, e: ex[l][e]))}
    x = torch.from_numpy(np.random.default_rng(5).standard_normal((80, moe.hidden))
                         .astype(np.float32)).cuda()
    toks = [token_id(gqa.seed, gqa.vocab, i) for i in range(80)]

    def run(kind):
        eng = engines[kind]
        if kind == "moe":
            return eng.prefill_layers(x)
        out = torch.empty((80, gqa.hidden), device="cuda")
        eng.prefill(toks, 0, x_out=out)
        return out

    yield run, {kind: run(kind).clone() for kind in engines}
    for eng in engines.values():
        eng.close()


@pytest.mark.parametrize("setting", SETTINGS)
@pytest.mark.parametrize("kind", ["gqa", "moe"])
def test_prefill_does_not_follow_global_precision_settings(stacks, kind, setting):
    run, want = stacks
    with SETTINGS[setting]():
        got = run(kind)
    assert torch.equal(got, want[kind])


@pytest.mark.parametrize("setting", [contextlib.nullcontext, tf32], ids=["", "tf32"])
@pytest.mark.parametrize("T,K,N", [(1, 512, 12), (33, 7168, 256)])
def test_the_routers_product_keeps_32_bits(T, K, N, setting):
    """Against 64 bits: three sums of K products each (2^-23 a product, as the matrix unit may
    cut), of x's three parts whose magnitudes add up to at most 1 + 2^-7 of x's, what the
    parts leave of x (2^-26) and the two additions of the sums."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn((T, K), generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-30, 30, (T, 1), generator=g, device="cuda"))
    w = torch.randn((N, K), generator=g, device="cuda").bfloat16()
    with setting():
        y = prefill._mm32(x, w)
    assert y.dtype == torch.float32
    ref, mag = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    tol = ((1 + 2 ** -7) * K * 2.0 ** -23 + 2.0 ** -26 + 2 * 2.0 ** -24) * mag
    assert ((y.double() - ref).abs() <= tol).all()
