"""The prompt path of an engine: T tokens at once through the stack the engine decodes, so
that its caches hold the prompt's keys and values before the first decode step.

Per layer, with the residual stream x in fp32 and the engine's own weights:

  x, xn = add_rmsnorm(x, previous sublayer's output);  q, k, v = Wq xn, Wk xn, Wv xn;
  rotate q and k at their positions; append k and v to the caches;
  o = prompt_attention(q, caches[0 .. pos + T));  x, hn = add_rmsnorm(x, Wo o);
  SwiGLU MLP, or the routed MXFP4 experts (mxfp4_matmul, rows grouped by expert).

The plain bf16 projections are library products.  Activations entering a product are bf16
(the decode step keeps them in fp32), sums and the residual stream fp32.  A prompt may be
run in pieces: each piece attends to what the caches already hold.  An application's settings
of matrix precision and autocast do not reach in here.  ``Engine.status()`` waits for a
prompt and tells whether its operators have finished their work.
"""
from __future__ import annotations

import torch

from . import ops, tre


def _refuse(status: int, msg: str):
    raise tre.TreError(status, "prefill", msg)


def _mm(x, w):
    """x [T][K] bf16 times w [N][K] bf16, transposed: [T][N] fp32."""
    return torch.mm(x, w.t(), out_dtype=torch.float32)


def _mm32(x, w):
    """x [T][K] fp32 times w [N][K] bf16, transposed, to fp32 accuracy whatever precision an
    application allows fp32 products: x as the sum of three bf16 numbers (8 of its 24 bits
    each), whose products with bf16 are exact in the fp32 sums."""
    high = x.bfloat16()
    rest = x - high
    middle = rest.bfloat16()
    return _mm(high, w) + (_mm(middle, w) + _mm((rest - middle).bfloat16(), w))


def _rotary(cfg, pos: int, T: int, device):
    """cos and sin [T][1][D / 2] of the angles p theta^(-2i/D): fp64 angles (a far position
    times a small frequency loses its fraction in fp32), fp32 values."""
    D = cfg.head_dim
    i = torch.arange(D // 2, dtype=torch.float64, device=device)
    p = torch.arange(pos, pos + T, dtype=torch.float64, device=device)
    ang = p[:, None] * torch.pow(float(cfg.rope_theta), -2.0 * i / D)[None, :]
    return ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]


def _rotate(v, cos, sin):
    """Half-split rotation of v [T][H][D] (fp32), rounded to bf16."""
    a, b = v.chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1).bfloat16()


def _swiglu(g, u):
    return (torch.nn.functional.silu(g) * u).bfloat16()


def _experts(cfg, w, x, hn):
    """Router, routed experts and shared experts of one MoE layer: [T][d] fp32."""
    T, d = x.shape
    E, k = cfg.n_experts, cfg.top_k
    # the router decides by order, so its input is the fp32 norm and not the bf16 one
    xn = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + cfg.norm_eps)
    scores = torch.sigmoid(_mm32(xn * w["ffn_norm"].float(), w["router"].view(E, d)))
    top, idx = torch.sort(scores, dim=-1, descending=True, stable=True)  # ties: lower index
    top, idx = top[:, :k], idx[:, :k]
    weight = top / top.sum(-1, keepdim=True)
    chosen, order = torch.sort(idx.reshape(-1), stable=True)
    offsets = torch.searchsorted(chosen, torch.arange(E + 1, device=x.device)).int()
    rows = hn[order // k]
    act = _swiglu(ops.mxfp4_matmul(rows, w["expert_gate"], offsets),
                  ops.mxfp4_matmul(rows, w["expert_up"], offsets))
    part = ops.mxfp4_matmul(act, w["expert_down"], offsets)
    back = torch.empty_like(order)
    back[order] = torch.arange(T * k, device=x.device)
    y = (part[back].view(T, k, d) * weight[..., None]).sum(1)
    if cfg.n_shared:
        y += _mm(_swiglu(_mm(hn, w["shared_gate"]), _mm(hn, w["shared_up"])), w["shared_down"])
    return y


def _weights(eng, layer: int) -> dict:
    cfg = eng.cfg
    moe = cfg.kind == tre.TRE_LAYER_MOE
    slots = tre.MOE_SLOTS if moe else tre.GQA_SLOTS
    w = eng.dev_model["layers"][layer]
    return {name: w[s] for name, s in slots.items() if s in w}


def _run(eng, x, pos: int, want_output: bool):
    cfg = eng.cfg
    T, d = x.shape
    Hq, Hkv, D = cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim
    cos, sin = _rotary(cfg, pos, T, x.device)
    delta = None
    for l in range(cfg.n_layers):
        w = _weights(eng, l)
        kc = eng.dev_model["k_cache"][l].view(Hkv, -1, D)
        vc = eng.dev_model["v_cache"][l].view(Hkv, -1, D)
        # the caller's x is not changed; from the second layer on x is ours, updated in place
        x, xn = ops.add_rmsnorm(x, delta, w["attn_norm"], cfg.norm_eps, x_out=x if l else None)
        k = _rotate(_mm(xn, w["wk"]).view(T, Hkv, D), cos, sin)
        v = _mm(xn, w["wv"]).view(T, Hkv, D)
        kc[:, pos:pos + T] = k.transpose(0, 1)
        vc[:, pos:pos + T] = v.transpose(0, 1)  # rounded to bf16 by the copy
        if l + 1 == cfg.n_layers and not want_output:
            return None
        q = _rotate(_mm(xn, w["wq"]).view(T, Hq, D), cos, sin)
        o = ops.prompt_attention(q, kc[:, :pos + T], vc[:, :pos + T])
        x, hn = ops.add_rmsnorm(x, _mm(o.view(T, Hq * D), w["wo"]), w["ffn_norm"], cfg.norm_eps,
                                x_out=x)
        if cfg.kind == tre.TRE_LAYER_MOE:
            delta = _experts(cfg, w, x, hn)
        else:
            delta = _mm(_swiglu(_mm(hn, w["wgate"]), _mm(hn, w["wup"])), w["wdown"])
    return x + delta


def _check(eng, T: int, pos: int) -> None:
    cfg = eng.cfg
    if cfg.kind == tre.TRE_LAYER_MLA:
        _refuse(tre.TRE_ERR_UNSUPPORTED, "MLA stacks have no prompt path")
    if cfg.kind == tre.TRE_LAYER_GQA and cfg.weight_format != tre.TRE_WEIGHTS_BF16:
        _refuse(tre.TRE_ERR_UNSUPPORTED, "GQA stacks run prompts with bf16 projections only")
    if cfg.kind == tre.TRE_LAYER_MOE and cfg.weight_format != tre.TRE_WEIGHTS_FP4_EXPERTS:
        _refuse(tre.TRE_ERR_UNSUPPORTED, "MoE stacks run prompts with MXFP4 experts only")
    if pos < 0 or pos + T > cfg.kv_capacity:
        _refuse(tre.TRE_ERR_POS_RANGE, f"positions [{pos}, {pos + T}) do not fit the cache of "
                                       f"{cfg.kv_capacity}")


def _out(x_out, x):
    if x_out is not None and (x_out.shape != x.shape or x_out.dtype != torch.float32 or
                              x_out.device != x.device):
        _refuse(tre.TRE_ERR_INVALID_ARG, "x_out must be fp32 [T][hidden] on the engine's device")


@torch.no_grad()
def prefill(eng, tokens, pos: int = 0, x_out=None) -> None:
    """Fill eng's caches with the keys and values of `tokens` at positions pos .. pos + T - 1
    (the caches hold [0, pos) on entry), enqueued on torch's current stream of the engine's
    device.  tokens: a list of ids, or a one-dimensional integer tensor (a device tensor's ids
    are read back once, to be checked against the vocabulary).  x_out (fp32 [T][hidden], optional)
    receives the residual stream after the last layer.  GQA stacks with bf16 projections and
    MoE stacks with MXFP4 experts."""
    cfg = eng.cfg
    if not cfg.has_embed_lm_head:
        _refuse(tre.TRE_ERR_INVALID_ARG, "a layers-only stack takes hidden vectors: "
                                         "prefill_layers")
    embed = eng.dev_model["embed"]
    if not isinstance(tokens, torch.Tensor):
        tokens = torch.tensor([int(t) for t in tokens], dtype=torch.int64)
    if tokens.ndim != 1 or tokens.is_floating_point() or tokens.dtype == torch.bool:
        _refuse(tre.TRE_ERR_INVALID_ARG, "tokens must be one-dimensional and whole numbers")
    T = tokens.numel()
    _check(eng, T, pos)
    if T and not (0 <= int(tokens.min()) and int(tokens.max()) < cfg.vocab):
        _refuse(tre.TRE_ERR_INVALID_ARG, f"a token is outside [0, {cfg.vocab})")
    if T == 0:
        return
    with torch.cuda.device(embed.device), torch.autocast("cuda", enabled=False):
        x = embed.view(cfg.vocab, cfg.hidden)[tokens.to(embed.device).long()].float()
        _out(x_out, x)
        y = _run(eng, x, pos, x_out is not None)
        if x_out is not None:
            x_out.copy_(y)


@torch.no_grad()
def prefill_layers(eng, x_in, pos: int = 0, x_out=None):
    """x_out [T][hidden] = the residual stream after the last layer of T consecutive positions
    from pos, from x_in (fp32 [T][hidden] on the engine's device), which is not changed;
    the caches then hold [0, pos + T)."""
    cfg = eng.cfg
    if x_in.ndim != 2 or x_in.shape[1] != cfg.hidden or x_in.dtype != torch.float32 or \
            not x_in.is_cuda or x_in.device != eng.dev_model["k_cache"][0].device:
        _refuse(tre.TRE_ERR_INVALID_ARG, "x_in must be fp32 [T][hidden] on the engine's device")
    _check(eng, x_in.shape[0], pos)
    _out(x_out, x_in)
    x_out = torch.empty_like(x_in) if x_out is None else x_out
    if x_in.shape[0]:
        with torch.cuda.device(x_in.device), torch.autocast("cuda", enabled=False):
            x_out.copy_(_run(eng, x_in.contiguous(), pos, True))
    return x_out
