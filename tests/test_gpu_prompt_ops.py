"""The prompt operators against plain implementations in 64 bits.

Tolerances, from half-step roundings (bf16 2^-8 relative, fp32 2^-24):

* attention: every probability is rounded to bf16 before the product with v (2^-8 p |v|);
  the fp32 score of D products and the exponential add less than 2^-10 of p (D 2^-24 times
  sums of |q k| scale under 2^6, exp2 to 2^-13), the output one bf16 rounding (2^-8 |o|).
* product: K fp32 additions in any order, counted at 2^-23 each (alignment inside the
  matrix unit may cut instead of round): K 2^-23 sum|x w|, plus the output's rounding.
* quantiser: exact.  Norm: fp32 sums of d squares ((d + 16) 2^-24 relative), bf16 output.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from persistent_tile_pipelined_b200 import ops, tre  # noqa: E402
from persistent_tile_pipelined_b200.synth import mxfp4_pitch  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert tre.tre_ops_status() == 0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)


# ---- attention ---------------------------------------------------------------------------------
def attention_ref(q, k, v, q_lens, kv_lens, scale):
    """(out, sum p |v|) in fp64: q [T, Hq, D], k, v [Hkv, S, D]."""
    T, Hq, D = q.shape
    g = Hq // k.shape[0]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    q0 = k0 = 0
    for nq, nk in zip(q_lens, kv_lens):
        kd = k[:, k0:k0 + nk].double().repeat_interleave(g, 0)
        vd = v[:, k0:k0 + nk].double().repeat_interleave(g, 0)
        for t in range(nq) if nq <= 64 else [None]:
            rows = slice(q0, q0 + nq) if t is None else slice(q0 + t, q0 + t + 1)
            ti = torch.arange(nq, device=q.device) if t is None else torch.tensor([t], device=q.device)
            see = torch.arange(nk, device=q.device)[None, :] <= (ti + nk - nq)[:, None]
            last = int(see.sum(-1).max()) if nk else 0
            if last == 0:
                continue
            s = torch.einsum("thd,hsd->hts", q[rows].double(), kd[:, :last]) * scale
            s = s.masked_fill(~see[:, :last], float("-inf"))
            p = torch.softmax(s, -1)
            p = torch.where(see[:, :last].any(-1)[:, None], p, 0.0)
            out[rows] = torch.einsum("hts,hsd->thd", p, vd[:, :last])
            mag[rows] = torch.einsum("hts,hsd->thd", p, vd[:, :last].abs())
        q0, k0 = q0 + nq, k0 + nk
    return out, mag


def check_attention(out, q, k, v, q_lens, kv_lens, scale=None):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    ref, mag = attention_ref(q, k, v, q_lens, kv_lens, scale)
    n = sum(q_lens)
    tol = (2 ** -8 + 2 ** -10) * mag + 2 ** -8 * ref.abs() + 1e-30
    err = (out.double() - ref).abs()[:n]
    bad = err > tol[:n]
    assert not bad.any() and out[:n].isfinite().all(), \
        f"{int(bad.sum())} of {bad.numel()} off, worst {float((err / tol[:n]).max()):.3g} of the tolerance"


SHAPES = [  # Hq, Hkv, D
    (4, 2, 64), (32, 8, 128), (7, 1, 128), (3, 3, 64), (40, 2, 128), (6, 2, 128)]
LENS = [  # one sequence over the cache layout: query rows, key rows
    (1, 1), (1, 129), (2, 2), (5, 300), (77, 205), (128, 128), (129, 129), (257, 700), (300, 120),
    (3, 4099), (1, 0)]


@pytest.mark.parametrize("nq,nk", LENS)
@pytest.mark.parametrize("hq,hkv,d", SHAPES)
def test_attention_one_sequence_over_a_cache(hq, hkv, d, nq, nk):
    g = gen(hq * 1000 + nq)
    q, k, v = normal(g, nq, hq, d), normal(g, hkv, nk + 40, d), normal(g, hkv, nk + 40, d)
    k[:, nk:], v[:, nk:] = float("nan"), float("inf")  # what lies behind the last key
    out = ops.prompt_attention(q, k[:, :nk], v[:, :nk])
    check_attention(out, q, k, v, [nq], [nk])


PACKED = [
    ([1, 1, 1], [1, 1, 1]), ([0, 5, 0, 130, 1, 0], [3, 5, 0, 130, 400, 0]),
    ([64, 200, 31], [64, 190, 500]), ([257, 1, 33], [300, 129, 20]), ([513, 511], [513, 1023]),
    ([1] * 33 + [100], list(range(0, 66, 2)) + [100])]


@pytest.mark.parametrize("q_lens,kv_lens", PACKED, ids=lambda x: str(len(x)))
@pytest.mark.parametrize("hq,hkv,d", SHAPES[:5])
def test_attention_packed(hq, hkv, d, q_lens, kv_lens):
    g = gen(hq + len(q_lens))
    T, S = sum(q_lens) + 3, sum(kv_lens) + 5  # rows of no sequence behind the last
    q = normal(g, T, hq, d)
    k, v = normal(g, S, hkv, d), normal(g, S, hkv, d)
    k[sum(kv_lens):], v[sum(kv_lens):] = float("nan"), float("nan")
    q[sum(q_lens):] = float("nan")
    out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    got = ops.prompt_attention(q, k.transpose(0, 1), v.transpose(0, 1), offsets(q_lens),
                               offsets(kv_lens), out=out)
    assert got is out
    check_attention(out, q, k.transpose(0, 1), v.transpose(0, 1), q_lens, kv_lens)
    assert (out[sum(q_lens):] == 7.0).all()


@pytest.mark.parametrize("hq,hkv,d,nq,nk", [(300, 1, 64, 5, 140), (1026, 2, 128, 2, 300),
                                            (257, 1, 128, 1, 1)])
def test_attention_more_heads_than_a_tile_has_rows(hq, hkv, d, nq, nk):
    g = gen(hq)
    q, k, v = normal(g, nq, hq, d), normal(g, hkv, nk, d), normal(g, hkv, nk, d)
    check_attention(ops.prompt_attention(q, k, v), q, k, v, [nq], [nk])


def test_attention_over_many_sequences():
    g = gen(9)
    q_lens = [(i * 7) % 23 for i in range(150)]
    kv_lens = [(i * 11) % 61 for i in range(150)]  # some shorter than their rows, some empty
    q = normal(g, sum(q_lens), 6, 64)
    k, v = normal(g, 2, sum(kv_lens), 64), normal(g, 2, sum(kv_lens), 64)
    out = ops.prompt_attention(q, k, v, offsets(q_lens), offsets(kv_lens))
    check_attention(out, q, k, v, q_lens, kv_lens)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_other_strides_and_scale(d):
    g = gen(5)
    T, hq, hkv = 150, 8, 2
    fused = normal(g, T, hq + 2 * hkv + 1, d + 8)[..., :d]
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv].transpose(0, 1), fused[:, hq + hkv:-1].transpose(0, 1)
    out = torch.zeros(T, hq + 1, d + 16, dtype=torch.bfloat16, device=DEV)
    ops.prompt_attention(q, k, v, scale=0.31, out=out[:, :hq, :d])
    check_attention(out[:, :hq, :d], q, k, v, [T], [T], 0.31)
    assert (out[:, hq:] == 0).all() and (out[..., d:] == 0).all()


@pytest.mark.parametrize("nq,nk", [(1, 33000), (4, 20011), (40, 9000)])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (4, 1, 64), (6, 2, 128)])
def test_attention_few_rows_over_many_keys(hq, hkv, d, nq, nk):
    g = gen(nk)
    q, k, v = normal(g, nq, hq, d), normal(g, hkv, nk, d), normal(g, hkv, nk, d)
    check_attention(ops.prompt_attention(q, k, v), q, k, v, [nq], [nk])


def test_attention_rows_keep_apart_what_they_do_not_see():
    """A key's NaN or infinity reaches the rows that see it and no other."""
    g = gen(11)
    for bad in (float("nan"), float("inf")):
        for at in (70, 130, 199):
            q, k, v = normal(g, 200, 4, 128), normal(g, 2, 200, 128), normal(g, 2, 200, 128)
            want = ops.prompt_attention(q[:at], k[:, :at], v[:, :at])
            for which in ("k", "v"):
                kk, vv = k.clone(), v.clone()
                (kk if which == "k" else vv)[:, at, 5] = bad
                out = ops.prompt_attention(q, kk, vv)
                assert torch.isfinite(out[:at]).all()
                ref, mag = attention_ref(q[:at], k[:, :at], v[:, :at], [at], [at], 128 ** -0.5)
                tol = (2 ** -8 + 2 ** -10) * mag + 2 ** -8 * ref.abs() + 1e-30
                assert ((out[:at].double() - ref).abs() <= tol).all()
                if which == "v":
                    assert not torch.isfinite(out[at:, :, 5]).any()
                    assert torch.isfinite(out[at:, :, 6]).all()
                elif bad != bad:
                    assert torch.isnan(out[at:]).all()
            assert want.shape == (at, 4, 128)


def test_attention_large_scores_and_equal_keys():
    g = gen(3)
    q, k, v = normal(g, 130, 8, 64, std=6.0), normal(g, 2, 400, 64, std=6.0), normal(g, 2, 400, 64)
    # scores reach ~1500: the fp32 product's error there is a share of the score, not of p
    out = ops.prompt_attention(q, k, v, scale=1.0)
    ref, mag = attention_ref(q, k, v, [130], [400], 1.0)
    sabs = torch.einsum("thd,hsd->hts", q.double().abs(),
                        k.double().abs().repeat_interleave(4, 0)).max()
    prel = 2 * float(sabs) * 64 * 2 ** -24 + 2 ** -8
    assert ((out.double() - ref).abs() <= 2 * prel * mag + 2 ** -8 * ref.abs() + 1e-30).all()
    k = k[:, :1].expand(2, 400, 64).contiguous()
    out = ops.prompt_attention(q, k, v)
    check_attention(out, q, k, v, [130], [400])


def test_attention_first_keys_score_far_below_later_ones():
    """The running maximum rises by thousands along the keys, and falls back."""
    g = gen(4)
    q = torch.ones(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(1, 1000, 64, dtype=torch.bfloat16, device=DEV)
    k[0, :, 0] = torch.linspace(-900, 900, 1000, device=DEV).bfloat16()
    k[0, 700:, 0] = -900.0
    v = normal(g, 1, 1000, 64)
    out = ops.prompt_attention(q, k, v, scale=1.0)
    check_attention(out, q, k, v, [3], [1000], 1.0)


def test_attention_offsets_outside_the_rows_are_clamped():
    g = gen(6)
    q, k, v = normal(g, 50, 4, 64), normal(g, 2, 60, 64), normal(g, 2, 60, 64)
    qo = torch.tensor([-7, 20, 1000], dtype=torch.int32, device=DEV)
    ko = torch.tensor([0, 30, 2000000000], dtype=torch.int32, device=DEV)
    check_attention(ops.prompt_attention(q, k, v, qo, ko), q, k, v, [20, 30], [30, 30])


def test_attention_same_bits_again_and_in_a_graph():
    g = gen(8)
    q, k, v = normal(g, 300, 32, 128), normal(g, 8, 3000, 128), normal(g, 8, 3000, 128)
    qo, ko = offsets([100, 1, 199]), offsets([500, 1500, 1000])
    first = ops.prompt_attention(q, k, v, qo, ko)
    assert torch.equal(first, ops.prompt_attention(q, k, v, qo, ko))
    few = ops.prompt_attention(q[:2], k, v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            ops.prompt_attention(q, k, v, qo, ko)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ops.prompt_attention(q, k, v, qo, ko)
        out2 = ops.prompt_attention(q[:2], k, v)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(out2, few)
    qo.copy_(offsets([7, 250, 43]))  # the captured call follows the offsets
    graph.replay()
    torch.cuda.synchronize()
    check_attention(out, q, k, v, [7, 250, 43], [500, 1500, 1000])


def test_attention_on_two_streams_at_once():
    g = gen(9)
    sets = [(normal(g, 2, 32, 128), normal(g, 8, 9000, 128), normal(g, 8, 9000, 128))
            for _ in range(2)]
    want = [ops.prompt_attention(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(ops.prompt_attention(*s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_attention_strides_beyond_32_bits():
    """Heads and rows that lie more than 2^31 elements apart."""
    g = gen(12)
    far = 2 ** 31 + 4096
    big = torch.empty(far + 2 ** 20, dtype=torch.bfloat16, device=DEV)
    k, v = (big.as_strided((2, 300, 64), (far, 128, 1), at) for at in (0, 64))
    k.copy_(normal(g, 2, 300, 64))
    v.copy_(normal(g, 2, 300, 64))
    q = normal(g, 140, 4, 64)
    check_attention(ops.prompt_attention(q, k, v), q, k, v, [140], [300])
    qf = big.as_strided((2, 4, 64), (far, 64, 1), 600 * 128)  # two rows, far apart
    qf.copy_(q[:2])
    of = big.as_strided((2, 4, 64), (far, 64, 1), 700 * 128)
    got = torch.empty_like(qf)
    ops.prompt_attention(qf, k, v, out=got)
    check_attention(got, q[:2], k, v, [2], [300])
    with pytest.raises(ValueError):  # the spans of out and the cache overlap
        ops.prompt_attention(qf, k, v, out=of)


@pytest.mark.parametrize("what", ["attention", "split", "product", "cluster", "quantize", "norm"])
def test_first_call_of_a_process_is_captured(what):
    """No operator needs a call before the one that a graph records."""
    import os
    import subprocess
    import sys
    code = """
import sys, torch
sys.path.insert(0, sys.argv[2])
from persistent_tile_pipelined_b200 import ops, tre
what = sys.argv[1]
r = lambda *s: torch.randn(s, device="cuda").bfloat16()
if what == "attention":
    q, k, v = r(200, 4, 64), r(2, 200, 64), r(2, 200, 64)
    f = lambda: ops.prompt_attention(q, k, v)
elif what == "split":
    q, k, v = r(1, 4, 128), r(2, 9000, 128), r(2, 9000, 128)
    f = lambda: ops.prompt_attention(q, k, v)
elif what in ("product", "cluster"):
    x = r(300 if what == "product" else 1, 1024)
    w = torch.randint(100, 120, (256, 544), dtype=torch.uint8, device="cuda")
    f = lambda: ops.mxfp4_matmul(x, w)
elif what == "quantize":
    w = r(64, 256)
    f = lambda: ops.mxfp4_dequantize(ops.mxfp4_quantize(w), 256)
else:
    x, g = torch.randn(9, 64, device="cuda"), r(64)
    f = lambda: ops.add_rmsnorm(x, None, g, 1e-5)[1]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = f()
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
assert torch.equal(out, f())
assert tre.tre_ops_status() == 0
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", code, what, root], capture_output=True, text=True,
                         timeout=120)
    assert run.returncode == 0 and "same" in run.stdout, run.stderr[-2000:]


def test_attention_refuses():
    g = gen(1)
    q, kv = normal(g, 5, 4, 64), normal(g, 2, 9, 64)
    with pytest.raises(ValueError):
        ops.prompt_attention(q, kv, kv[:, :8])
    with pytest.raises(ValueError):
        ops.prompt_attention(q, kv, kv, offsets([5]))
    with pytest.raises(ValueError):
        ops.prompt_attention(q, kv, kv, offsets([5]).long(), offsets([9]))
    with pytest.raises(ValueError):
        ops.prompt_attention(q, kv, kv, out=q)
    with pytest.raises(ValueError, match="gradient"):
        ops.prompt_attention(q.clone().requires_grad_(), kv, kv)
    with pytest.raises(tre.TreError) as e:
        ops.prompt_attention(normal(g, 5, 3, 64), kv, kv)
    assert e.value.status == tre.TRE_ERR_INVALID_ARG
    with pytest.raises(tre.TreError):
        ops.prompt_attention(q, kv[:1].expand(2, 9, 64), kv)


# ---- MXFP4 rows --------------------------------------------------------------------------------
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def quantize_ref(w):
    """Scale bytes and codes of w [R, K] (fp64), from the definition."""
    b = w.reshape(w.shape[0], -1, 32)
    top = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where(bad, 1.0, top))) - 2
    byte = np.where(top == 0, 0, np.clip(e + 127, 0, 254)).astype(int)
    a = np.abs(np.where(bad[..., None], 0.0, b)) * 2.0 ** (127.0 - byte[..., None])
    dist = np.abs(np.minimum(a, 6.0)[..., None] - GRID)
    near = dist.min(-1, keepdims=True) == dist
    code = np.where(near & (np.arange(8) % 2 == 0), np.arange(8), -1).max(-1)  # the even one
    code = np.where(code >= 0, code, near.argmax(-1))
    code = code + 8 * (np.signbit(b) & ~bad[..., None])
    return np.where(bad, 255, byte), code.reshape(w.shape)


def unpack(rows, K):
    rows = rows.cpu().numpy()
    codes = np.stack([rows[:, :K // 2] & 15, rows[:, :K // 2] >> 4], -1).reshape(len(rows), K)
    return rows[:, K // 2:K // 2 + K // 32].astype(int), codes, rows[:, K // 2 + K // 32:]


def decoded(rows, K):
    byte, codes, _ = unpack(rows, K)
    val = GRID[codes & 7] * np.where(codes >= 8, -1.0, 1.0)
    scale = np.where(byte == 255, np.nan, 2.0 ** (byte - 127.0))
    return val * np.repeat(scale, 32, -1)


def weights(R, K, dtype, seed=0):
    """Values of every kind: ordinary ones, ties, groups of zeros, huge and tiny groups, values
    just above a power of two, signed zeros."""
    g = gen(seed)
    w = torch.randn((R, K // 32, 32), generator=g, device=DEV)
    scale = torch.randint(-20, 20, (R, K // 32, 1), generator=g, device=DEV)
    ties = torch.randint(-28, 29, (R, K // 32, 32), generator=g, device=DEV) / 4.0
    kind = torch.randint(0, 6, (R, K // 32, 1), generator=g, device=DEV)
    w = torch.where(kind == 1, ties, w)
    w = torch.where(kind == 2, w * 2.0 ** scale, w)
    w = torch.where(kind == 3, torch.zeros_like(w).copysign(w), w)
    w = torch.where(kind == 4, w * 2.0 ** -125.0, w)  # subnormals among them
    w = torch.where(kind == 5, w.clamp(-3, 3) * 2.0 ** 126.0, w)
    return w.reshape(R, K).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (7, 96), (130, 544), (33, 2048), (5, 7168)])
def test_quantize_is_exact(R, K, dtype):
    w = weights(R, K, dtype, R + K)
    rows = ops.mxfp4_quantize(w)
    assert rows.shape == (R, mxfp4_pitch(K)) and rows.dtype == torch.uint8
    byte, codes, pad = unpack(rows, K)
    want_byte, want_codes = quantize_ref(w.double().cpu().numpy())
    assert (byte == want_byte).all()
    assert (codes == want_codes).all()
    assert (pad == 0).all()
    for out_dtype in (torch.bfloat16, torch.float32):
        back = ops.mxfp4_dequantize(rows, K, out_dtype).double().cpu().numpy()
        assert (back == decoded(rows, K)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_quantize_a_long_matrix_like_its_parts(dtype):
    """Over a million groups take another form of the kernels than the parts do."""
    w = weights(4099, 8256, dtype, 5)
    rows = ops.mxfp4_quantize(w)
    parts = [ops.mxfp4_quantize(p) for p in w.split(1000)]
    assert torch.equal(rows, torch.cat(parts))
    for out_dtype in (torch.bfloat16, torch.float32):
        back = ops.mxfp4_dequantize(rows, 8256, out_dtype)
        assert torch.equal(back, torch.cat([ops.mxfp4_dequantize(p, 8256, out_dtype)
                                            for p in parts]))


def test_quantize_strides_batches_and_bad_values():
    w = weights(24, 64, torch.float32, 1)
    wide = torch.zeros(24, 80, device=DEV)
    wide[:, :64] = w
    want = ops.mxfp4_quantize(w)
    assert torch.equal(ops.mxfp4_quantize(wide[:, :64]), want)
    for at, pad in ((4, 20), (8, 16), (4, 24)):  # rows at 16 bytes of every 32, or some of them
        off = torch.zeros(24, 64 + pad, device=DEV)[:, at:at + 64]
        off.copy_(w)
        assert torch.equal(ops.mxfp4_quantize(off), want)
        half = torch.zeros(24, 64 + 2 * pad, device=DEV, dtype=torch.bfloat16)[:, 2 * at:2 * at + 64]
        half.copy_(w)
        assert torch.equal(ops.mxfp4_quantize(half), ops.mxfp4_quantize(w.bfloat16()))
    assert torch.equal(ops.mxfp4_quantize(w.view(2, 3, 4, 64)), want.view(2, 3, 4, -1))
    assert torch.equal(ops.mxfp4_quantize(w[0]), want[0])
    out = torch.full((26, mxfp4_pitch(64)), 9, dtype=torch.uint8, device=DEV)
    ops.mxfp4_quantize(w, out=out[1:25])
    assert torch.equal(out[1:25], want) and (out[0] == 9).all() and (out[25] == 9).all()
    for bad in (float("nan"), float("inf"), -float("inf")):
        w2 = w.clone()
        w2[3, 40] = bad
        rows = ops.mxfp4_quantize(w2)
        byte, codes, _ = unpack(rows, 64)
        assert byte[3, 1] == 255 and (codes[3, 32:] == 0).all()
        rows[3] = want[3]
        assert torch.equal(rows, want)
        back = ops.mxfp4_dequantize(ops.mxfp4_quantize(w2), 64)
        assert torch.isnan(back[3, 32:]).all() and torch.isfinite(back[3, :32]).all()
    assert ops.mxfp4_quantize(w[:0]).shape == (0, mxfp4_pitch(64))


def test_dequantize_every_code_and_scale():
    rows = torch.zeros((256, 32), dtype=torch.uint8, device=DEV)
    rows[:, :16] = torch.arange(16, device=DEV, dtype=torch.uint8)[None] * 16 + \
        torch.arange(15, -1, -1, device=DEV, dtype=torch.uint8)[None]
    rows[:, 16] = torch.arange(256, device=DEV, dtype=torch.int32).to(torch.uint8)
    want = decoded(rows, 32)
    with np.errstate(over="ignore"):
        for dt in (torch.bfloat16, torch.float32):
            back = ops.mxfp4_dequantize(rows, 32, dt).double().cpu().numpy()
            top = want.astype(np.float32).astype(np.float64)
            assert np.array_equal(back, top, equal_nan=True)


# ---- product -----------------------------------------------------------------------------------
def matmul_case(T, E, R, K, lens, seed=0, x_pad=0):
    g = gen(seed + T + R)
    w = ops.mxfp4_quantize(normal(g, E, R, K, std=0.02))
    x = normal(g, T, K + x_pad)[:, :K]
    return x, w, None if lens is None else offsets(lens)


def check_matmul(y, x, w, lens, K):
    E, R = w.shape[0], w.shape[1]
    wd = torch.from_numpy(decoded(w.view(E * R, -1), K)).to(DEV).view(E, R, K)
    row = 0
    half = torch.finfo(y.dtype).eps / 2
    for e, c in enumerate([x.shape[0]] if lens is None else lens):
        if c:
            xe = x[row:row + c].double()
            ref, mag = xe @ wd[e].t(), xe.abs() @ wd[e].abs().t()
            tol = K * 2.0 ** -23 * mag + half * ref.abs() + 1e-30
            err = (y[row:row + c].double() - ref).abs()
            assert (err <= tol).all(), f"expert {e}: {float((err / tol).max()):.3g} of the tolerance"
        row += c


MATMULS = [  # T, E, R, K, rows of each expert
    (1, 1, 128, 32, None), (1, 1, 2048, 7168, None), (3, 1, 7, 64, None), (16, 1, 130, 416, None),
    (17, 1, 129, 992, None), (200, 1, 300, 736, None), (515, 1, 1000, 2080, None),
    (33, 4, 200, 256, [0, 1, 32, 0]), (150, 3, 65, 160, [0, 150, 0]),
    (700, 5, 260, 544, [300, 7, 129, 0, 264]), (8, 8, 512, 1024, [1] * 8),
    (90, 40, 48, 96, [0, 9] * 10 + [0] * 20), (2100, 2, 136, 320, [1050, 1050])]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("T,E,R,K,lens", MATMULS, ids=lambda x: str(x) if isinstance(x, int) else "")
def test_matmul(T, E, R, K, lens, dtype):
    x, w, off = matmul_case(T, E, R, K, lens)
    y = ops.mxfp4_matmul(x, w, off, dtype)
    assert y.shape == (T, R) and y.dtype == dtype
    check_matmul(y, x, w, lens, K)
    assert torch.equal(y, ops.mxfp4_matmul(x, w, off, dtype))


# more experts than a lane's 32 loads cover, most of them without rows
@pytest.mark.parametrize("T,E", [(300, 257), (2500, 1100)])
def test_matmul_many_experts(T, E):
    lens = [0] * E
    for i in range(T):
        lens[(i * 97 + i // 50) % E if i % 3 else E - 1 - i % 5] += 1
    x, w, off = matmul_case(T, E, 40, 96, lens)
    check_matmul(ops.mxfp4_matmul(x, w, off), x, w, lens, 96)


# tiles of 256 rows, more of them than SMs: a CTA takes several, whose steps and copies of
# weights end at odd places
MANY = [(600, 1, 9000, 64, None), (1030, 4, 5100, 96, [257, 0, 513, 260]),
        (2000, 3, 6500, 352, [1, 1500, 499]), (700, 2, 9600, 1312, [700, 0])]


@pytest.mark.parametrize("T,E,R,K,lens", MANY, ids=lambda x: str(x) if isinstance(x, int) else "")
def test_matmul_several_tiles_a_cta(T, E, R, K, lens):
    x, w, off = matmul_case(T, E, R, K, lens)
    y = ops.mxfp4_matmul(x, w, off, torch.bfloat16)
    check_matmul(y, x, w, lens, K)
    assert torch.equal(y, ops.mxfp4_matmul(x, w, off, torch.bfloat16))


def test_matmul_on_two_streams_at_once():
    cases = [matmul_case(16, 1, 512, 2048, None, seed=i) for i in range(2)]
    cases += [matmul_case(600, 1, 9000, 64, None, seed=i) for i in range(2)]
    want = [ops.mxfp4_matmul(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(ops.mxfp4_matmul(*c))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_matmul_large_and_small_scales_in_one_row():
    """Scales on both sides of 1 (byte 127) and beyond 2 (128), mixed within rows and between
    the rows of a warp."""
    T, R, K = 20, 140, 512
    x, w, _ = matmul_case(T, 1, R, K, None)
    g = gen(2)
    w[0, :, K // 2:K // 2 + K // 32] = torch.randint(100, 150, (R, K // 32), generator=g, device=DEV,
                                                     dtype=torch.int32).to(torch.uint8)
    w[0, 7::32, K // 2:] = 120  # rows without a large one
    check_matmul(ops.mxfp4_matmul(x, w), x, w, None, K)


def test_matmul_rows_of_no_expert_strides_and_bad_neighbours():
    lens, K, R = [5, 0, 40], 128, 200
    x, w, _ = matmul_case(60, 3, R, K, lens, x_pad=8)
    off = offsets([4] + lens)[1:].contiguous()  # the first 4 rows belong to none
    x[:4], x[49:] = float("nan"), float("inf")
    x[4 + 5:4 + 6] = float("nan")  # one row of the last expert
    out = torch.full((60, R + 3), 5.0, device=DEV)
    ops.mxfp4_matmul(x, w, off, out=out[:, :R])
    assert (out[:4] == 5).all() and (out[49:] == 5).all() and (out[:, R:] == 5).all()
    assert torch.isnan(out[9, :R]).all()
    check_matmul(out[4:9, :R], x[4:9], w[:1], None, K)
    check_matmul(out[10:49, :R], x[10:49], w[2:], None, K)


def test_matmul_scales_of_every_size():
    """Scale bytes from 0 to 254: exact products of one code and one activation each; byte
    255 stands for NaN and spoils its own matrix row only."""
    K, R = 64, 256
    w = torch.zeros((1, R, mxfp4_pitch(K)), dtype=torch.uint8, device=DEV)
    w[0, :, 3] = 0x30  # element 7: 1.5
    w[0, :, 20] = 0x0a  # element 40: -1.0
    w[0, :, K // 2] = torch.arange(256, device=DEV, dtype=torch.int32).to(torch.uint8)
    w[0, :, K // 2 + 1] = 127
    x = torch.zeros((1, K), dtype=torch.bfloat16, device=DEV)
    x[0, 7] = 1.0
    y = ops.mxfp4_matmul(x, w)[0].double().cpu()
    want = 1.5 * 2.0 ** (torch.arange(256, dtype=torch.float64) - 127)
    normal_ = (want >= 2.0 ** -126) & (torch.arange(256) < 255)
    assert torch.equal(y[normal_], want[normal_])
    assert (y[want < 2.0 ** -126] <= 2.0 ** -126).all() and torch.isnan(y[255])
    x[0, 7], x[0, 40] = 0.0, 2.0
    y = ops.mxfp4_matmul(x, w)[0]
    assert (y[:255] == -2.0).all() and torch.isnan(y[255])


def test_matmul_offsets_are_clamped_and_read_on_the_device():
    x, w, _ = matmul_case(40, 2, 96, 64, None)
    off = torch.tensor([-3, 10, 4000], dtype=torch.int32, device=DEV)
    check_matmul(ops.mxfp4_matmul(x, w, off), x, w, [10, 30], 64)
    off = offsets([20, 20])
    ops.mxfp4_matmul(x, w, off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.mxfp4_matmul(x, w, off)
    for lens in ([20, 20], [0, 40], [33, 7]):
        off.copy_(offsets(lens))
        graph.replay()
        torch.cuda.synchronize()
        check_matmul(y, x, w, lens, 64)


def test_matmul_refuses():
    x, w, off = matmul_case(10, 2, 64, 64, [5, 5])
    with pytest.raises(ValueError):
        ops.mxfp4_matmul(x, w)
    with pytest.raises(ValueError):
        ops.mxfp4_matmul(x, w, off[:2])
    with pytest.raises(ValueError):
        ops.mxfp4_matmul(x.float(), w, off)
    with pytest.raises(ValueError):
        ops.mxfp4_matmul(x, w[..., :32], off)
    with pytest.raises(ValueError):
        ops.mxfp4_matmul(x, w, off, torch.float16)
    with pytest.raises(tre.TreError):
        ops.mxfp4_matmul(torch.zeros(10, 68, dtype=torch.bfloat16, device=DEV)[:, 2:66], w, off)


# ---- residual addition and norm ----------------------------------------------------------------
@pytest.mark.parametrize("T,d", [(1, 8), (1, 4096), (3, 264), (70, 7168), (2, 9000), (2, 40000),
                                 (1500, 4104), (1100, 520), (2, 20008), (1, 32768)])
@pytest.mark.parametrize("delta", [None, torch.bfloat16, torch.float32], ids=str)
def test_add_rmsnorm(T, d, delta):
    g = gen(T + d)
    x = normal(g, T, d, dtype=torch.float32)
    dl = None if delta is None else normal(g, T, d, dtype=delta)
    gain = (1 + normal(g, d, dtype=torch.float32, std=0.01)).bfloat16()
    keep = x.clone()
    xo, out = ops.add_rmsnorm(x, dl, gain, 1e-5)
    assert torch.equal(x, keep)
    want_x = x if dl is None else x + dl.float()
    assert torch.equal(xo, want_x)
    xd = want_x.double()
    ref = xd / torch.sqrt(xd.square().mean(-1, keepdim=True) + 1e-5) * gain.double()
    tol = (2 ** -8 + (d + 16) * 2.0 ** -24) * ref.abs() + 1e-30
    assert ((out.double() - ref).abs() <= tol).all()
    # in place, and on rows of wider tensors
    wide = torch.zeros(T, d + 8, device=DEV)
    wide[:, :d] = x
    xi, out2 = ops.add_rmsnorm(wide[:, :d], dl, gain, 1e-5, x_out=wide[:, :d])
    assert torch.equal(wide[:, :d], want_x) and torch.equal(out2, out)
    assert (wide[:, d:] == 0).all()


def test_add_rmsnorm_zero_rows_and_bad_values():
    gain = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    x = torch.zeros(5, 64, device=DEV)
    x[2, 3] = float("nan")
    x[3, 3] = float("inf")
    xo, out = ops.add_rmsnorm(x, None, gain, 1e-6)
    assert (out[[0, 1, 4]] == 0).all() and torch.isnan(out[2]).all()
    assert torch.isnan(out[3, 3]) and (out[3, :3] == 0).all()
    big = torch.full((1, 64), 1e15, device=DEV)
    assert (ops.add_rmsnorm(big, None, gain, 1e-6)[1] == 1).all()
    assert ops.add_rmsnorm(x[:0], None, gain, 1e-6)[1].shape == (0, 64)
    with pytest.raises(ValueError):
        ops.add_rmsnorm(x, x, gain, 1e-6, x_out=x)
    with pytest.raises(ValueError):
        ops.add_rmsnorm(x, None, gain[:32], 1e-6)
    with pytest.raises(tre.TreError):
        ops.add_rmsnorm(x, None, gain, -1.0)
