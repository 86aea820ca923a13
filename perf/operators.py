"""Cases of the prompt operators: attention over prompts, the MXFP4 rows of the experts with
their product, and the residual addition with its RMS norm.

Where ``own`` is false every operator runs in its plain form (elementary torch operations in
32 bits, rounded once); where it is true the same cases run through
``persistent_tile_pipelined_b200.ops``.

A case is a dict of plain values with its ``op``:

* ``attention``: ``hq`` query heads over ``hkv`` key/value heads of width ``d``; sequence i
  has ``q[i]`` query rows over ``kv[i]`` cached rows (both as texts of numbers).
* ``quantize``: ``e`` matrices of ``r`` rows of ``k`` weights of type ``type``, to MXFP4 rows
  and back to the values that these stand for.
* ``product``: ``t`` rows of ``k`` activations, spread over ``e`` experts of ``r`` output
  rows each (``route`` seeds the spread; ``e`` = 1: all rows), result of type ``type``.
* ``norm``: ``t`` rows of ``d``, a ``delta`` of that type (or "none") added before the norm.
"""
import math
import random

import torch

own = False


def listed():
    return [
        # a chunk of a prompt against the cache of the repository's tiny stack: launch latency
        dict(name="attn-tiny-chunk", op="attention", hq=4, hkv=2, d=64, q="77", kv="205"),
        # one token of the 8B-shaped stack over its longest cache: the bytes of the cache
        dict(name="attn-token-131072", op="attention", hq=32, hkv=8, d=128, q="1", kv="131072"),
        # prompts of many lengths packed behind each other, one of them on a cached prefix, a
        # one-token one, an empty one and one whose first rows see no key
        dict(name="attn-packed", op="attention", hq=64, hkv=8, d=128,
             q="1031,333,1,0,1500,129,517,40", kv="1031,333,1,0,2777,129,517,25"),
        # the 8192-token prompt of the 8B-shaped stack: the matrix units
        dict(name="attn-prompt-8192", op="attention", hq=32, hkv=8, d=128, q="8192", kv="8192"),
        # one expert's gate matrix, as a loader takes them one by one
        dict(name="quantize-expert", op="quantize", e=1, r=2048, k=7168, type="bf16"),
        # a stack of trained fp32 experts of an odd row count
        dict(name="quantize-stack-f32", op="quantize", e=24, r=1999, k=7168, type="f32"),
        # one row through one expert: latency, the bytes of one matrix
        dict(name="product-1row", op="product", t=1, e=1, r=2048, k=7168, route=0, type="f32"),
        # a short prompt's rows in a few experts, odd sizes
        dict(name="product-ragged", op="product", t=403, e=12, r=1000, k=736, route=5, type="bf16"),
        # 512 tokens x top-8 over the MoE layer's 256 experts, gate projection: the bytes of W
        dict(name="product-moe-gate", op="product", t=4096, e=256, r=2048, k=7168, route=1,
             type="bf16"),
        # a long prompt in a few large experts, down projection: the matrix units
        dict(name="product-long-down", op="product", t=8192, e=4, r=7168, k=2048, route=2,
             type="f32"),
        # one row of the 8B-shaped stack
        dict(name="norm-1row", op="norm", t=1, d=4096, delta="bf16"),
        # a long prompt of the MoE stack, expert sums added in fp32
        dict(name="norm-8192", op="norm", t=8192, d=7168, delta="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "quantize", "product", "product", "norm"])
    if op == "attention":
        hkv, g, d = rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 4, 7, 8, 16]), rng.choice([64, 128])
        form = rng.choice(["token", "chunk", "packed", "packed"])
        if form == "token":
            q, kv = [rng.randint(1, 4)], [_log(rng, 5, 131072)]
        elif form == "chunk":
            q = [_log(rng, 2, 3000)]
            kv = [q[0] + _log(rng, 1, 4096)]
        else:
            n = rng.randint(2, 12)
            q = [_log(rng, 1, 5000 // n) for _ in range(n)]
            kv = [a + rng.choice([0, 0, 0, -1, 1, rng.randint(1, 300)]) for a in q]
        while len(q) > 1 and hkv * g * sum(q) * sum(kv) > 2 ** 31:
            q, kv = q[:-1], kv[:-1]
        while hkv * g * sum(q) * sum(kv) > 2 ** 31:
            g = max(1, g // 2)
            q = [max(1, a // 2) for a in q]
        return dict(op=op, hq=hkv * g, hkv=hkv, d=d, q=",".join(map(str, q)),
                    kv=",".join(map(str, kv)))
    if op == "quantize":
        k = 32 * _log(rng, 1, 256)
        return dict(op=op, e=rng.randint(1, 6), r=_log(rng, 1, 3000), k=k,
                    type=rng.choice(["bf16", "f32"]))
    if op == "product":
        e = rng.choice([1, 1, 3, 8, 30])
        return dict(op=op, t=_log(rng, 1, 5000), e=e, r=_log(rng, 8, 5000), k=32 * _log(rng, 1, 160),
                    route=rng.randint(0, 999), type=rng.choice(["bf16", "f32"]))
    return dict(op=op, t=_log(rng, 1, 8192), d=8 * _log(rng, 8, 1024),
                delta=rng.choice(["bf16", "f32", "none"]))


def _lens(text):
    return [int(a) for a in text.split(",")]


def _offsets(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _counts(case):
    """Rows of each expert: a skewed spread, some experts without a row."""
    t, e = case["t"], case["e"]
    if e == 1:
        return [t]
    rng = random.Random(case["route"])
    weight = [rng.random() ** 2 for _ in range(e)]
    counts = [0] * e
    for i in rng.choices(range(e), weights=weight, k=t):
        counts[i] += 1
    return counts


def _pitch(k):
    return (k // 2 + k // 32 + 15) // 16 * 16


def _type(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        out = torch.empty(shape, dtype=dtype, device="cuda")
        return out.normal_(mean, std, generator=g)

    op = case["op"]
    if op == "attention":
        q, kv = _lens(case["q"]), _lens(case["kv"])
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        one = len(q) == 1  # one prompt over the engine's cache layout; else packed rows
        state = dict(case, scale=1.0 / math.sqrt(d), q=normal(sum(q), hq, d))
        if one:
            cap = sum(kv) + 64
            state["k"] = normal(hkv, cap, d)[:, :sum(kv)]
            state["v"] = normal(hkv, cap, d)[:, :sum(kv)]
            state["q_offsets"] = state["kv_offsets"] = None
        else:
            state["k"] = normal(sum(kv), hkv, d).transpose(0, 1)
            state["v"] = normal(sum(kv), hkv, d).transpose(0, 1)
            for key, lens in (("q_offsets", q), ("kv_offsets", kv)):
                state[key] = torch.tensor(_offsets(lens), dtype=torch.int32, device="cuda")
        return state
    if op == "quantize":
        return dict(case, w=normal(case["e"], case["r"], case["k"], std=0.02,
                                   dtype=_type(case["type"])))
    if op == "product":
        e, r, k = case["e"], case["r"], case["k"]
        w = torch.zeros((e, r, _pitch(k)), dtype=torch.uint8, device="cuda")
        w[..., :k // 2].random_(0, 256, generator=g)
        w[..., k // 2:k // 2 + k // 32].random_(119, 121, generator=g)
        counts = _counts(case)
        return dict(case, x=normal(case["t"], k), w=w, most=max(counts),
                    offsets=None if e == 1 else torch.tensor(_offsets(counts), dtype=torch.int32,
                                                             device="cuda"))
    t, d = case["t"], case["d"]
    return dict(case, eps=1e-5, x=normal(t, d, dtype=torch.float32),
                delta=None if case["delta"] == "none" else normal(t, d, dtype=_type(case["delta"])),
                gain=normal(d, mean=1.0, std=0.01))


def run(state):
    op = state["op"]
    if own:
        from persistent_tile_pipelined_b200 import ops
        if op == "attention":
            return ops.prompt_attention(state["q"], state["k"], state["v"], state["q_offsets"],
                                        state["kv_offsets"])
        if op == "quantize":
            return ops.mxfp4_dequantize(ops.mxfp4_quantize(state["w"]), state["k"])
        if op == "product":
            return ops.mxfp4_matmul(state["x"], state["w"], state["offsets"],
                                    out_dtype=_type(state["type"]))
        return ops.add_rmsnorm(state["x"], state["delta"], state["gain"], state["eps"])
    if op == "attention":
        return _attention(state)
    if op == "quantize":
        return _round_trip(state["w"])
    if op == "product":
        return _product(state)
    x = state["x"] if state["delta"] is None else state["x"] + state["delta"].float()
    norm = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + state["eps"])
    return x, (norm * state["gain"].float()).bfloat16()


def _attention(s):
    """softmax(scale q k^T) v over every pair of rows, those of no sequence in common or of a
    later position left out; rows without a key are zero."""
    q, k, v = s["q"], s["k"], s["v"]
    (t, hq, d), (hkv, n, _) = q.shape, k.shape
    qi, ki = torch.arange(t, device=q.device), torch.arange(n, device=q.device)
    if s["q_offsets"] is None:
        see = ki[None, :] <= qi[:, None] + (n - t)
    else:
        qo, ko = s["q_offsets"].long(), s["kv_offsets"].long()
        qs = torch.searchsorted(qo[1:], qi, right=True)
        ks = torch.searchsorted(ko[1:], ki, right=True)
        last = qi - qo[qs + 1] + ko[qs + 1]
        see = (qs[:, None] == ks[None, :]) & (ki[None, :] <= last[:, None])
    rows = q.float().view(t, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)
    p = torch.bmm(rows, k.float().transpose(1, 2)).mul_(s["scale"]).view(hkv, -1, t, n)
    p.masked_fill_(~see, -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p.view(hkv, -1, n), v.float()).view(hkv, -1, t, d)
    out = torch.where(total > 0, out / total, 0.0)
    return out.permute(2, 0, 1, 3).reshape(t, hq, d).bfloat16()


def _round_trip(w):
    """The values that w's MXFP4 rows stand for, a bf16 number each."""
    b = w.float().unflatten(-1, (-1, 32))
    _, e = torch.frexp(b.abs().amax(-1, keepdim=True))  # max = m 2^e, m in [0.5, 1)
    e = (e - 3).clamp_(-127, 127)
    a = torch.ldexp(b.abs(), -e).clamp_(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step  # round() takes ties to the even multiple
    return torch.copysign(torch.ldexp(a, e), b).flatten(-2).bfloat16()


def _decode(w, k):
    """The numbers that MXFP4 rows of k elements stand for, in 32 bits."""
    codes = w[..., :k // 2]
    codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    a = (codes & 7).float()
    a = torch.where(a < 4, a * 0.5, torch.where(a < 6, a - 2.0, a * 2.0 - 8.0))
    a = torch.where(codes < 8, a, -a)
    scale = torch.exp2(w[..., k // 2:k // 2 + k // 32].float() - 127.0)
    return a.unflatten(-1, (-1, 32)).mul_(scale[..., None]).flatten(-2)


def _product(s):
    """The rows of each expert, filled up to the largest count, times its decoded matrix."""
    x, offsets = s["x"].float(), s["offsets"]
    w = _decode(s["w"], s["k"])
    if offsets is None:
        return (x @ w[0].t()).to(_type(s["type"]))
    t = torch.arange(x.shape[0], device=x.device)
    expert = torch.searchsorted(offsets[1:].long(), t, right=True)
    place = t - offsets.long()[expert]
    rows = x.new_zeros(w.shape[0], s["most"], x.shape[1])
    rows[expert, place] = x
    return torch.bmm(rows, w.transpose(1, 2))[expert, place].to(_type(s["type"]))


def work(case):
    op = case["op"]
    if op == "attention":
        q, kv, hq, hkv, d = (_lens(case["q"]), _lens(case["kv"]), case["hq"], case["hkv"],
                             case["d"])
        pairs = read = 0
        for a, b in zip(q, kv):
            first = b - a + 1  # keys that the first row sees; below 1: rows without a key
            lo = max(first, 1)
            pairs += (lo + b) * (b - lo + 1) // 2 if b >= lo else 0
            read += b if a else 0
        return {"bytes": 2 * d * (2 * hq * sum(q) + 2 * hkv * read), "flops": 4 * d * hq * pairs}
    if op == "quantize":
        n, k = case["e"] * case["r"], case["k"]
        size = 2 if case["type"] == "bf16" else 4
        return {"bytes": n * (k * (size + 2) + 2 * _pitch(k)), "flops": 0}
    if op == "product":
        t, r, k = case["t"], case["r"], case["k"]
        used = sum(c > 0 for c in _counts(case))
        size = 2 if case["type"] == "bf16" else 4
        return {"bytes": used * r * _pitch(k) + t * (2 * k + size * r), "flops": 2 * t * r * k}
    t, d = case["t"], case["d"]
    delta = {"bf16": 2, "f32": 4, "none": 0}[case["delta"]]
    return {"bytes": t * d * (4 + delta + 4 + 2) + 2 * d, "flops": 6 * t * d}


def exact(case, seed):
    """The definitions, sequence by sequence and expert by expert, in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "attention":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        q0 = k0 = 0
        for nq, nk in zip(_lens(case["q"]), _lens(case["kv"])):
            blind = max(0, nq - nk)  # the first rows, which see nothing
            for h in range(hq if nq > blind else 0):
                kh = s["k"][h * hkv // hq, k0:k0 + nk].double()
                vh = s["v"][h * hkv // hq, k0:k0 + nk].double()
                logits = s["q"][q0 + blind:q0 + nq, h].double() @ kh.t() / math.sqrt(d)
                hide = torch.ones_like(logits, dtype=torch.bool).triu(1 + nk - (nq - blind))
                logits[hide] = -math.inf
                out[q0 + blind:q0 + nq, h] = torch.softmax(logits, -1) @ vh
            q0, k0 = q0 + nq, k0 + nk
        return out
    if op == "quantize":
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        middle = (grid[1:] + grid[:-1]) / 2
        outs = []
        for w in s["w"]:
            b = w.double().unflatten(-1, (-1, 32))
            top = b.abs().amax(-1, keepdim=True)
            scale = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -126))) - 2)
            a = b.abs() / scale
            near = torch.bucketize(a, middle)  # a value in the middle goes to the lower one
            tie = (a == middle[near.clamp(max=6)]) & (near % 2 == 1) & (near < 7)
            outs.append((grid[near + tie] * scale * torch.sign(b)).flatten(-2).float())
        return torch.stack(outs)
    if op == "product":
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        table = torch.cat([table, -table])
        x, k = s["x"], case["k"]
        out = torch.zeros((case["t"], case["r"]), dtype=torch.float64, device="cuda")
        row = 0
        for e, c in enumerate(_counts(case)):
            if c:
                w = s["w"][e]
                m = torch.empty((case["r"], k), dtype=torch.float64, device="cuda")
                m[:, 0::2] = table[(w[:, :k // 2] % 16).int()]
                m[:, 1::2] = table[(w[:, :k // 2] // 16).int()]
                power = w[:, k // 2:k // 2 + k // 32].double() - 127
                m *= torch.pow(2.0, power).repeat_interleave(32, 1)
                out[row:row + c] = x[row:row + c].double() @ m.t()
            row += c
        return out
    x = s["x"].double()
    if s["delta"] is not None:
        x = x + s["delta"].double()
    r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + s["eps"])
    return x, x * r * s["gain"].double()
