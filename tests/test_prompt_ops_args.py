"""Refusals of the prompt operators: what a C caller can get wrong is refused on the host,
before anything is enqueued (no GPU needed: the addresses are never touched)."""
import ctypes

import pytest

from persistent_tile_pipelined_b200 import build

build.build_engine()
from persistent_tile_pipelined_b200 import tre  # noqa: E402

INVALID = tre.TRE_ERR_INVALID_ARG
P = 1 << 20  # a 16-byte aligned address


def attention(**over):
    a = tre.tre_attention(8, 2, 128, 0, 5, 9, 8 * 128, 128, 128, 9 * 128, 128, 9 * 128, 8 * 128,
                          128, 0.088)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def test_attention_descriptor_is_accepted_by_the_workspace_query():
    assert tre.tre_prompt_attention_workspace(attention()) >= 0
    assert tre.tre_prompt_attention_workspace(attention(n_q_rows=0)) == 0


@pytest.mark.parametrize("over", [
    dict(head_dim=96), dict(head_dim=0), dict(n_kv_heads=0), dict(n_q_heads=0),
    dict(n_q_heads=7), dict(n_seqs=-1), dict(n_q_rows=-1), dict(n_kv_rows=-3),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(q_row_stride=1028), dict(k_row_stride=4), dict(v_head_stride=-128),
    dict(out_head_stride=127), dict(k_row_stride=0), dict(out_row_stride=64),
    dict(out_row_stride=256, out_head_stride=128), dict(n_q_rows=1 << 28), dict(n_kv_rows=(1 << 30) + 1),
], ids=str)
def test_attention_refuses(over):
    a = attention(**over)
    b = ctypes.c_size_t()
    assert tre.lib.tre_prompt_attention_workspace(ctypes.byref(a), 148, ctypes.byref(b)) == INVALID
    assert tre.lib.tre_last_error()
    assert tre.tre_prompt_attention(a, P, P, P, 0, 0, P) == INVALID


@pytest.mark.parametrize("args", [
    (0, P, P, 0, 0, P), (P, 0, P, 0, 0, P), (P, P, P + 8, 0, 0, P), (P + 2, P, P, 0, 0, P),
    (P, P, P, 0, 0, 0)], ids=str)
def test_attention_refuses_pointers(args):
    assert tre.tre_prompt_attention(attention(), *args) == INVALID


def test_attention_refuses_sequences_without_offsets_and_a_short_workspace():
    assert tre.tre_prompt_attention(attention(n_seqs=2), P, P, P, 0, P, P) == INVALID
    assert tre.tre_prompt_attention(attention(n_seqs=2), P, P, P, P, P + 2, P) == INVALID
    long = attention(n_q_rows=1, n_kv_rows=100000)
    need = tre.tre_prompt_attention_workspace(long)
    if need:
        assert tre.tre_prompt_attention(long, P, P, P, 0, 0, P, P, need - 1) == INVALID
        assert tre.tre_prompt_attention(long, P, P, P, 0, 0, P, 0, 0) == INVALID


def test_nothing_to_do_is_accepted():
    assert tre.tre_prompt_attention(attention(n_q_rows=0), 0, 0, 0, 0, 0, 0) == tre.TRE_OK
    assert tre.tre_mxfp4_quantize(0, tre.TRE_BF16, 0, 32, 32, 0) == tre.TRE_OK
    assert tre.tre_mxfp4_dequantize(0, 0, 64, tre.TRE_F32, 0) == tre.TRE_OK
    assert tre.tre_mxfp4_matmul(0, 32, 0, 0, 1, 0, 8, 32, tre.TRE_F32, 0, 8) == tre.TRE_OK
    assert tre.tre_add_rmsnorm(0, 8, 0, 0, 0, 0, 1e-5, 0, 8, 0, 8, 0, 8) == tre.TRE_OK


@pytest.mark.parametrize("args", [
    (P, 2, 4, 64, 64, P), (P, 0, -1, 64, 64, P), (P, 0, 4, 48, 64, P), (P, 0, 4, 0, 64, P),
    (0, 0, 4, 64, 64, P), (P, 0, 4, 64, 64, 0), (P + 4, 0, 4, 64, 64, P), (P, 0, 4, 64, 64, P + 1),
    (P, 0, 4, 64, 68, P), (P, 1, 4, 64, 66, P), (P, 0, 4, 64, -64, P)], ids=str)
def test_quantize_refuses(args):
    assert tre.tre_mxfp4_quantize(*args) == INVALID


@pytest.mark.parametrize("args", [
    (P, 4, 64, 7, P), (P, -4, 64, 0, P), (P, 4, 40, 0, P), (0, 4, 64, 0, P), (P, 4, 64, 0, P + 4)],
    ids=str)
def test_dequantize_refuses(args):
    assert tre.tre_mxfp4_dequantize(*args) == INVALID


def matmul(**over):
    a = dict(x=P, x_row_stride=64, w=P, offsets=P, n_experts=3, rows=5, n=9, k=64,
             out_type=tre.TRE_F32, out=P, out_row_stride=9)
    a.update(over)
    return tre.tre_mxfp4_matmul(**a)


@pytest.mark.parametrize("over", [
    dict(out_type=2), dict(n_experts=0), dict(n_experts=1 << 17), dict(offsets=0),
    dict(offsets=P + 2), dict(rows=-1), dict(rows=1 << 30), dict(n=0), dict(n=1 << 30),
    dict(k=48), dict(k=0), dict(x=0), dict(x=P + 8), dict(w=0), dict(w=P + 8), dict(out=0),
    dict(out=P + 2), dict(x_row_stride=68), dict(x_row_stride=56), dict(out_row_stride=8)],
    ids=str)
def test_matmul_refuses(over):
    assert matmul(**over) == INVALID
    assert tre.lib.tre_last_error().startswith(b"tre_mxfp4_matmul")


def norm(**over):
    a = dict(x=P, x_row_stride=64, delta=P, delta_type=tre.TRE_BF16, delta_row_stride=64, gain=P,
             eps=1e-5, rows=5, d=64, x_out=P, x_out_row_stride=64, out=P, out_row_stride=64)
    a.update(over)
    return tre.tre_add_rmsnorm(**a)


@pytest.mark.parametrize("over", [
    dict(rows=-1), dict(d=0), dict(d=60), dict(eps=-1.0), dict(eps=float("nan")),
    dict(delta_type=3), dict(x=0), dict(gain=0), dict(out=0), dict(x=P + 4), dict(delta=P + 8),
    dict(x_out=P + 8), dict(x_row_stride=66), dict(delta_row_stride=68), dict(out_row_stride=56),
    dict(x_out_row_stride=60), dict(x_row_stride=128)], ids=str)
def test_norm_refuses(over):
    assert norm(**over) == INVALID


def test_torch_level_refusals_on_cpu_tensors():
    torch = pytest.importorskip("torch")
    from persistent_tile_pipelined_b200 import ops
    h = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    kv = torch.zeros(2, 6, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.prompt_attention(h, kv, kv)
    with pytest.raises(ValueError, match="type"):
        ops.prompt_attention(h.float(), kv, kv)
    with pytest.raises(ValueError, match="dimensions"):
        ops.prompt_attention(h[0], kv, kv)
    with pytest.raises(ValueError, match="CUDA"):
        ops.mxfp4_quantize(torch.zeros(4, 64))
    with pytest.raises(ValueError, match="type"):
        ops.mxfp4_quantize(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA"):
        ops.mxfp4_dequantize(torch.zeros(4, 48, dtype=torch.uint8), 64)
    with pytest.raises(ValueError, match="CUDA"):
        ops.mxfp4_matmul(torch.zeros(4, 64, dtype=torch.bfloat16),
                         torch.zeros(8, 48, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        ops.add_rmsnorm(torch.zeros(4, 64), None, torch.zeros(64, dtype=torch.bfloat16), 1e-5)


def test_the_attention_descriptor_matches_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lines = ['#include <stdio.h>', '#include "tre.h"', 'int main(void) {',
             'printf("%zu %d %d", sizeof(tre_attention), TRE_BF16, TRE_F32);']
    lines += [f'printf(" %zu", offsetof(tre_attention, {f}));' for f, _ in
              tre.tre_attention._fields_]
    src = tmp_path / "probe.c"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.check_call([cc, "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o",
                           str(tmp_path / "probe")])
    got = subprocess.run([str(tmp_path / "probe")], capture_output=True, text=True,
                         check=True).stdout
    want = [ctypes.sizeof(tre.tre_attention), tre.TRE_BF16, tre.TRE_F32]
    want += [getattr(tre.tre_attention, f).offset for f, _ in tre.tre_attention._fields_]
    assert [int(a) for a in got.split()] == want
