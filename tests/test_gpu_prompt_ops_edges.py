"""The prompt operators at the ends of their ranges, against the definitions in 64 bits."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from persistent_tile_pipelined_b200 import ops, tre  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    assert tre.tre_ops_status() == 0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


# ---- attention: scores of every finite size ------------------------------------------------
def attention_ref(q, k, v, scale):
    """(out, sum p |v|, scores) in fp64 of one sequence: q [T, Hq, D], k, v [Hkv, S, D]."""
    T, S, g = q.shape[0], k.shape[1], q.shape[1] // k.shape[0]
    s = torch.einsum("thd,hsd->hts", q.double(), k.double().repeat_interleave(g, 0)) * scale
    see = torch.arange(S, device=DEV)[None] <= torch.arange(T, device=DEV)[:, None] + S - T
    s = s.masked_fill(~see, float("-inf"))
    p = torch.where(see, torch.softmax(s, -1), 0.0)
    vd = v.double().repeat_interleave(g, 0)
    return (torch.einsum("hts,hsd->thd", p, vd), torch.einsum("hts,hsd->thd", p, vd.abs()), s)


# The forms of the kernel: two row tiles, one that two warpgroups share, keys split over CTAs.
FORMS = [(200, 260, 8, 2, 128), (3, 700, 4, 2, 64), (1, 9000, 8, 2, 128), (2, 5000, 4, 1, 64)]

# q . k = 2^e x + 2^(e - b) j with x of a few bits and whole j, exact in fp32; e + log2(scale):
# from ordinary scores over those whose base-2 logarithm passes 2^24 to the end of fp32.
SIZES = [(10, 6, 1.0), (25, 23, 1.0), (25, 23, 2.0), (26, 23, 1.0), (30, 22, 1.0), (31, 22, 1.0),
         (33, 20, 1.0), (40, 22, 1.0), (45, 22, 2.0 ** -10), (100, 22, 1.0), (125, 22, 1.0),
         (126, 20, 2.0 ** -100)]


def sized(g, nq, nk, hq, hkv, d, e, b, order):
    """q, k, v with scores as above; x falls, rises or varies along the keys."""
    top = e // 2
    q = torch.zeros(nq, hq, d, device=DEV)
    q[..., 0], q[..., 1] = 2.0 ** top, 2.0 ** (e - b - (e - b) // 2)
    q[1::3] *= -1.0  # rows whose scores are all negative
    q[2::4, :, :2] = 0.0  # rows whose scores are all zero
    k = torch.zeros(hkv, nk, d, device=DEV)
    x = 1.0 + torch.randint(0, 4, (hkv, nk), generator=g, device=DEV) / 4.0
    if order == "ties":
        x = torch.ones_like(x)
    elif order != "any":
        x = x.sort(-1, descending=order == "falls").values
    j = torch.randint(-3, 4, (hkv, nk), generator=g, device=DEV).float()
    k[..., 0] = x * 2.0 ** (e - top)
    k[..., 1] = j * 2.0 ** ((e - b) // 2)
    return q.bfloat16(), k.bfloat16(), normal(g, hkv, nk, d)


@pytest.mark.parametrize("order", ["any", "rises", "falls", "ties"])
@pytest.mark.parametrize("e,b,scale", SIZES)
@pytest.mark.parametrize("nq,nk,hq,hkv,d", FORMS)
def test_attention_scores_of_every_size(nq, nk, hq, hkv, d, e, b, scale, order):
    """The scores are exact, so what is left are the roundings of ordinary ones: p's to bf16
    (2^-8) and its exponential (2^-13; the exponent's own rounding is 2^-24 of at most 150, and
    of 150 2^-24 for the factor scale log2(e)), the output's (2^-8)."""
    q, k, v = sized(gen(e + nq), nq, nk, hq, hkv, d, e, b, order)
    out = ops.prompt_attention(q, k, v, scale=scale)
    ref, mag, _ = attention_ref(q, k, v, scale)
    assert out.isfinite().all()
    tol = (2 ** -8 + 2 ** -10) * mag + 2 ** -8 * ref.abs() + 1e-30
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), f"{int((err > tol).sum())} of {err.numel()}, {float((err / tol).max()):.3g}"


@pytest.mark.parametrize("bad", [False, True], ids=["finite", "nan-behind"])
@pytest.mark.parametrize("std", [2e4, 6e4, 1e9, 1e17])
@pytest.mark.parametrize("nq,nk,hq,hkv,d", FORMS)
def test_attention_large_random_scores(nq, nk, hq, hkv, d, std, bad):
    """Rows whose best score leads by more than what fp32 products can be off (2^-23 a product
    of the sum of magnitudes, on either side) and 40: the best key's value."""
    g = gen(int(std) % 1000 + nq)
    q, k = normal(g, nq, hq, d, std=std), normal(g, hkv, nk, d, std=std)
    v = normal(g, hkv, nk, d)
    scale = d ** -0.5
    if bad:  # the last key's value spoils the last row's result, and the rows go the long way
        v[:, -1, 3] = float("nan")
    out = ops.prompt_attention(q, k, v, scale=scale)
    _, _, s = attention_ref(q, k, torch.zeros_like(v), scale)
    mag = torch.einsum("thd,hsd->hts", q.double().abs(),
                       k.double().abs().repeat_interleave(hq // hkv, 0)) * scale
    best, at = s.topk(2, -1)
    lead = (best[..., 0] - best[..., 1]) > 2 * d * 2.0 ** -23 * mag.amax(-1) + 40
    assert lead[:, :nq].float().mean() > 0.5
    vd = v.double().repeat_interleave(hq // hkv, 0)
    want = torch.stack([vd[h, at[h, :, 0]] for h in range(hq)], 1)  # [T, Hq, D]
    keep = lead.t()
    if bad:
        keep[-1] = False
        assert out[-1, :, 3].isnan().all()
        out = out[:-1]
        keep, want = keep[:-1], want[:-1]
    assert out.isfinite().all()
    if keep.any():
        err = (out.double() - want).abs()[keep]
        assert (err <= 2 * 2.0 ** -8 * want[keep].abs() + 1e-15).all()


@pytest.mark.parametrize("e", [10, 33, 100])
@pytest.mark.parametrize("near", [3, 7])
def test_attention_rows_of_one_warp_with_scores_of_different_sizes(near, e):
    """Token 71 is the first of its eight to see the second key tile: with 4 heads a kv head the
    32 rows of a warp, which end their large rows before the small ones (near 7) or not."""
    g = gen(e)
    q, k, v = sized(g, 200, 257, 8, 2, 64, e, 20, "any")
    q[near::8] = normal(g, 25, 8, 64)
    k[..., 2:] = normal(g, 2, 257, 62)  # which the large rows do not look at
    q[near::8, :, :2] = 0.0
    out = ops.prompt_attention(q, k, v, scale=0.5)
    ref, mag, _ = attention_ref(q, k, v, 0.5)
    tol = (2 ** -8 + 2 ** -10) * mag + 2 ** -8 * ref.abs() + 1e-30
    assert ((out.double() - ref).abs() <= tol).all()


# ---- errors of earlier calls -----------------------------------------------------------------
def every_operator(g):
    """A call of each operator, as functions."""
    q, kv = normal(g, 5, 4, 64), normal(g, 2, 9, 64)
    far = normal(g, 2, 9000, 64)
    x, w = normal(g, 3, 64), normal(g, 8, 64)
    rows = ops.mxfp4_quantize(w)
    r, gain = normal(g, 3, 64, dtype=torch.float32), normal(g, 64)
    return {"attention": lambda: ops.prompt_attention(q, kv, kv),
            "split": lambda: ops.prompt_attention(q[:1], far, far),
            "quantize": lambda: ops.mxfp4_quantize(w),
            "dequantize": lambda: ops.mxfp4_dequantize(rows, 64),
            "product": lambda: ops.mxfp4_matmul(x, rows),
            "norm": lambda: ops.add_rmsnorm(r, None, gain, 1e-5)[1]}


@pytest.mark.parametrize("op", ["attention", "split", "quantize", "dequantize", "product", "norm"])
def test_an_earlier_error_of_the_caller_is_not_the_operators(op):
    """The runtime keeps a thread's last failed call until it is asked for: an operator that is
    enqueued neither reports it nor takes it from the caller."""
    runtime = ctypes.CDLL("libcudart.so.12")  # the one that torch and libtre.so have loaded
    call = every_operator(gen(1))[op]
    want = call()
    runtime.cudaGetLastError()
    failed = runtime.cudaSetDevice(9999)  # refused on the host
    assert failed != 0
    got = call()
    assert runtime.cudaGetLastError() == failed and runtime.cudaGetLastError() == 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("op", ["attention", "split", "quantize", "product", "norm"])
def test_forward_mode_gradients_are_refused(op):
    """No operator has derivatives: an input with a tangent is refused like one that requires a
    gradient."""
    from torch.autograd import forward_ad
    g = gen(2)
    q, kv = normal(g, 5, 4, 64), normal(g, 2, 9, 64)
    far = normal(g, 2, 9000, 64)
    x, w = normal(g, 3, 64), normal(g, 8, 64)
    r, gain = normal(g, 3, 64, dtype=torch.float32), normal(g, 64)
    rows = ops.mxfp4_quantize(w)
    call, inputs = {
        "attention": (ops.prompt_attention, (q, kv, kv)),
        "split": (ops.prompt_attention, (q[:1], far, far)),
        "quantize": (ops.mxfp4_quantize, (w,)),
        "product": (lambda a: ops.mxfp4_matmul(a, rows), (x,)),
        "norm": (lambda a, b, c: ops.add_rmsnorm(a, b, c, 1e-5), (r, x, gain))}[op]
    with forward_ad.dual_level():
        call(*inputs)
        for i, t in enumerate(inputs):
            dual = forward_ad.make_dual(t, torch.ones_like(t))
            with pytest.raises(ValueError, match="gradient"):
                call(*inputs[:i], dual, *inputs[i + 1:])
    with pytest.raises(ValueError, match="gradient"):
        torch.func.jvp(lambda a: call(a, *inputs[1:]), (inputs[0],), (inputs[0],))


# ---- attention: infinite scores -----------------------------------------------------------------
@pytest.mark.parametrize("slow", [False, True], ids=["", "bad-value-behind"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")], ids=str)
@pytest.mark.parametrize("nq,nk,hq,hkv,d", FORMS)
def test_attention_infinite_scores(nq, nk, hq, hkv, d, bad, slow):
    """A row that sees a score of +infinity or NaN is NaN; one of -infinity has no weight."""
    g = gen(nq + nk)
    q, k, v = normal(g, nq, hq, d), normal(g, hkv, nk, d), normal(g, hkv, nk, d)
    at = nk - 1 - nq // 2
    k[:, at, 5] = bad
    q[..., 5] = torch.where(q[..., 5] == 0, 1.0, q[..., 5])
    if slow:  # the last key's value spoils the last row's result, and the rows go the long way
        v[:, -1, 3] = float("nan")
    out = ops.prompt_attention(q, k, v)
    _, _, s = attention_ref(q, k, torch.zeros_like(v), d ** -0.5)  # [hq, nq, nk]
    poisoned = ((s == float("inf")) | s.isnan()).any(-1).t()  # [nq, hq]
    assert poisoned.any() or bad == -float("inf") or nq < 4
    assert out[poisoned].isnan().all()
    p = torch.softmax(s.masked_fill(poisoned.t()[..., None], 0.0), -1)
    vd = v.double().repeat_interleave(hq // hkv, 0)
    if slow:
        assert out[-1, :, 3].isnan().all()
        vd[:, -1, 3] = 0.0  # compared below without the last row
    ref, mag = (torch.einsum("hts,hsd->thd", p, a) for a in (vd, vd.abs()))
    ok = ~poisoned
    if slow:
        ok[-1] = False
    tol = (2 ** -8 + 2 ** -10) * mag + 2 ** -8 * ref.abs() + 1e-30
    assert ((out.double() - ref).abs() <= tol)[ok].all()


@pytest.mark.parametrize("nq,nk,hq,hkv,d", FORMS)
def test_attention_rows_of_minus_infinite_scores_alone(nq, nk, hq, hkv, d):
    """The definition's 0 / 0: a row that sees nothing else is NaN in every form."""
    q = torch.ones(nq, hq, d, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(hkv, nk, d, dtype=torch.bfloat16, device=DEV)
    k[..., 0] = -float("inf")
    v = normal(gen(nk), hkv, nk, d)
    assert ops.prompt_attention(q, k, v).isnan().all()


# ---- product: the smallest weights ---------------------------------------------------------------
@pytest.mark.parametrize("T", [1, 20, 40, 100, 300])
def test_matmul_is_exact_with_the_smallest_scales(T):
    """Weights below 2^-126 (numbers that bf16 holds with fewer bits) times 2^64: exact."""
    K, R = 64, 16 * 8
    w = torch.zeros((1, R, (K // 2 + K // 32 + 15) // 16 * 16), dtype=torch.uint8, device=DEV)
    code = torch.arange(R, device=DEV) % 16
    byte = torch.arange(R, device=DEV) // 16  # 0 .. 7
    w[0, :, 3] = (code << 4).to(torch.uint8)  # element 7
    w[0, :, K // 2] = byte.to(torch.uint8)
    w[0, :, K // 2 + 1] = 127
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    x[:, 7] = 2.0 ** 64
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    want = grid[code % 8] * torch.where(code < 8, 1.0, -1.0).double() * 2.0 ** (byte - 127.0 + 64)
    y = ops.mxfp4_matmul(x, w).double()
    assert (y == want[None]).all()


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (6, 1, 64)])
def test_attention_of_a_decode_batch(hq, hkv, d):
    """One token of each of several sequences over caches of very different lengths, some of them
    empty: the keys are split, and each sequence ends in another part."""
    g = gen(hq)
    lens = [20000, 1, 0, 129, 7000, 128]
    q = normal(g, len(lens) + 2, hq, d)  # two rows in front that belong to no sequence
    k, v = normal(g, sum(lens), hkv, d).transpose(0, 1), normal(g, sum(lens), hkv, d).transpose(0, 1)
    ends = torch.tensor([0] + lens, device=DEV).cumsum(0).int()
    rows = torch.arange(2, len(lens) + 3, device=DEV, dtype=torch.int32)
    out = torch.full_like(q, 7.0)
    ops.prompt_attention(q, k, v, rows, ends, out=out)
    assert (out[:2] == 7.0).all()
    at = 0
    for i, n in enumerate(lens):
        if n == 0:
            assert (out[2 + i] == 0).all()
            continue
        ref, mag, _ = attention_ref(q[2 + i:3 + i], k[:, at:at + n], v[:, at:at + n], d ** -0.5)
        tol = (2 ** -8 + 2 ** -10) * mag + 2 ** -8 * ref.abs() + 1e-30
        assert ((out[2 + i:3 + i].double() - ref).abs() <= tol).all()
        at += n
