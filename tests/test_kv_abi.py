"""Host validation and struct layouts of the 8-bit KV cache calls (no GPU):
every refusal returns before any CUDA call, and the pointers are fake."""
import ctypes
import os
import subprocess

import pytest

from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli, synth

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20            # a fake, aligned address (never dereferenced)
INVALID, UNSUPPORTED, RESIDUAL, WORKSPACE, ALIGNMENT = 1, 2, 4, 5, 6


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return qli.lib()


@pytest.mark.parametrize("c_name,mirror", [("qli_kv_attn_args", qli.KVAttnArgs),
                                           ("qli_merge_args", qli.MergeArgs)])
def test_struct_layout_matches_header(tmp_path, c_name, mirror):
    fields = [f for f, _ in mirror._fields_]
    src = ['#include <stddef.h>', '#include <stdio.h>', '#include "qli.h"', 'int main(void){',
           'printf("%%zu\\n", sizeof(%s));' % c_name]
    src += ['printf("%%zu\\n", offsetof(%s, %s));' % (c_name, f) for f in fields]
    src += ['return 0;}']
    c = tmp_path / "probe.c"
    c.write_text("\n".join(src))
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(exe)], check=True)
    vals = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                           check=True).stdout.split()]
    assert vals[0] == ctypes.sizeof(mirror)
    for f, off in zip(fields, vals[1:]):
        assert getattr(mirror, f).offset == off, f


PAGE = dict(pages=10, stride=41216, R=64, ko=0, so=32768)
PAGE_REJECT = [
    (dict(n=-1), INVALID), (dict(x=None), INVALID), (dict(slot=None), INVALID),
    (dict(cache=None), INVALID), (dict(pages=-1), INVALID), (dict(R=32), UNSUPPORTED),
    (dict(quant=3), UNSUPPORTED), (dict(ko=41216 - 64 * 512 + 16), INVALID),
    (dict(so=41216 - 128 + 2), INVALID), (dict(ko=-16), INVALID), (dict(so=-2), INVALID),
    (dict(stride=0), INVALID), (dict(x_stride=504), INVALID), (dict(x_stride=516), ALIGNMENT),
    (dict(x=P + 8), ALIGNMENT), (dict(cache=P + 8), ALIGNMENT), (dict(stride=41224), ALIGNMENT),
    (dict(ko=8), ALIGNMENT), (dict(so=32769), ALIGNMENT), (dict(slot=P + 4), ALIGNMENT),
    (dict(err=P + 2), ALIGNMENT),
]


def _rows(L, which, **kw):
    a = dict(PAGE, x=P, x_stride=512, n=4, slot=P, cache=P, quant=2, err=None)
    a.update(kw)
    if which == "write":
        return L.qli_write_kv(a["x"], a["x_stride"], a["n"], a["slot"], a["cache"], a["pages"],
                              a["stride"], a["R"], a["ko"], a["so"], a["quant"], a["err"], None)
    return L.qli_read_kv(a["cache"], a["pages"], a["stride"], a["R"], a["ko"], a["so"], a["quant"],
                         a["slot"], a["n"], a["x"], a["x_stride"], a["err"], None)


@pytest.mark.parametrize("which", ["write", "read"])
@pytest.mark.parametrize("over,want", PAGE_REJECT)
def test_row_calls_refuse(L, which, over, want):
    assert _rows(L, which, **over) == want


@pytest.mark.parametrize("which", ["write", "read"])
def test_no_rows_is_nothing_to_do(L, which):
    assert _rows(L, which, n=0, x=None, slot=None, cache=None) == qli.OK


def good_attn(listed=True, **over):
    a = qli.KVAttnArgs()
    a.q = P; a.q_stride_t = 64 * 512; a.q_stride_h = 512
    a.T, a.H, a.D = 4, 64, 512
    a.cu_seqlens_q = P; a.B = 2
    a.cache = P; a.page_stride = 82432; a.num_pages = 100; a.rows_per_page = 128
    a.quant_mode = 2; a.kv_offset = 0; a.kv_scale_offset = 65536
    a.block_table = P; a.bt_stride = 8
    a.scale = 0.044
    if listed:
        a.indices = P; a.K = 256
    else:
        a.k_lens = P; a.ratio = 1
    a.out = P; a.out_stride_t = 64 * 512; a.out_stride_h = 512
    a.lse = P
    for k, v in over.items():
        setattr(a, k, v)
    return a


ATTN_REJECT = [
    (dict(D=576), UNSUPPORTED), (dict(H=0), UNSUPPORTED), (dict(H=129), UNSUPPORTED),
    (dict(rows_per_page=32), UNSUPPORTED), (dict(quant_mode=0), UNSUPPORTED),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(T=-1), INVALID), (dict(B=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(bt_stride=0), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(cache=None), INVALID), (dict(block_table=None), INVALID), (dict(cu_seqlens_q=None), INVALID),
    (dict(kv_offset=16912), INVALID), (dict(kv_scale_offset=82432 - 254), INVALID),
    (dict(kv_offset=-16), INVALID), (dict(q_stride_h=504), INVALID), (dict(out_stride_t=8), INVALID),
    (dict(q=P + 8), ALIGNMENT), (dict(q_stride_h=516), ALIGNMENT), (dict(out=P + 2), ALIGNMENT),
    (dict(out_stride_h=516), ALIGNMENT), (dict(page_stride=82440), ALIGNMENT),
    (dict(kv_offset=8), ALIGNMENT), (dict(kv_scale_offset=65537), ALIGNMENT),
    (dict(lse=P + 2), ALIGNMENT), (dict(err_word=P + 1), ALIGNMENT),
]
LISTED_REJECT = [(dict(K=0), INVALID), (dict(window=5), INVALID), (dict(indices=P + 2), ALIGNMENT)]
DENSE_REJECT = [(dict(k_lens=None), INVALID), (dict(ratio=0), UNSUPPORTED), (dict(ratio=4), UNSUPPORTED),
                (dict(residual=P), RESIDUAL), (dict(window=-1), INVALID), (dict(k_lens=P + 2), ALIGNMENT)]


@pytest.mark.parametrize("listed,over,want",
                         [(m, o, w) for m in (True, False) for o, w in ATTN_REJECT] +
                         [(True, o, w) for o, w in LISTED_REJECT] +
                         [(False, o, w) for o, w in DENSE_REJECT])
def test_attention_refuses(L, listed, over, want):
    a = good_attn(listed, **over)
    n = ctypes.c_size_t(0)
    assert L.qli_kv_attention(ctypes.byref(a), P, 1 << 40, None) == want
    assert L.qli_kv_attention_workspace_size(ctypes.byref(a), ctypes.byref(n)) == want


def test_attention_nothing_to_do(L):
    a = good_attn(T=0)
    assert L.qli_kv_attention(ctypes.byref(a), None, 0, None) == qli.OK
    assert L.qli_kv_attention(None, None, 0, None) == INVALID


def good_merge(parts=2, **over):
    a = qli.MergeArgs()
    a.parts, a.T, a.H, a.D = parts, 4, 64, 512
    for i in range(min(parts, qli.MERGE_MAX)):
        a.part_out[i] = P; a.part_lse[i] = P
        a.part_stride_t[i] = 64 * 512; a.part_stride_h[i] = 512
    a.out = P; a.out_stride_t = 64 * 512; a.out_stride_h = 512
    a.lse = P
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,want", [
    (dict(parts=0), INVALID), (dict(parts=5), INVALID), (dict(D=256), UNSUPPORTED),
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(out=None), INVALID),
    (dict(out=P + 8), ALIGNMENT), (dict(out_stride_h=4), INVALID), (dict(out_stride_t=516), ALIGNMENT),
    (dict(lse=P + 2), ALIGNMENT)])
def test_merge_refuses(L, over, want):
    assert L.qli_merge_attention(ctypes.byref(good_merge(**over)), None) == want


def test_merge_refuses_bad_parts(L):
    call = lambda a: L.qli_merge_attention(ctypes.byref(a), None)  # noqa: E731
    a = good_merge(); a.part_out[1] = None
    assert call(a) == INVALID
    a = good_merge(); a.part_lse[0] = None
    assert call(a) == INVALID
    a = good_merge(); a.part_out[1] = P + 8
    assert call(a) == ALIGNMENT
    a = good_merge(); a.part_stride_h[1] = 516
    assert call(a) == ALIGNMENT
    a = good_merge(parts_f32=1); a.part_stride_h[1] = 516      # 16 bytes of FP32
    a.T = 0
    assert call(a) == qli.OK
    a = good_merge(); a.part_stride_t[0] = -8
    assert call(a) == INVALID
    assert call(good_merge(T=0)) == qli.OK


def test_binding_refuses_host_and_mistyped_tensors():
    torch = pytest.importorskip("torch")
    geom = dict(rows_per_page=64, page_stride=41216, kv_offset=0, kv_scale_offset=32768)
    x = torch.zeros(2, 512, dtype=torch.bfloat16)
    slots, cache = torch.zeros(2, dtype=torch.int64), torch.zeros(1, 41216, dtype=torch.uint8)
    with pytest.raises(TypeError):
        qli.write_kv(x, slots, cache, **geom)
    with pytest.raises(TypeError):
        qli.read_kv(cache, slots, **geom)
    with pytest.raises(TypeError):
        qli.kv_attention(x[None], slots, cache, slots, scale=1.0, **geom)
    with pytest.raises(ValueError):
        qli.merge_attention([], [])
    with pytest.raises(TypeError):
        qli.merge_attention([torch.zeros(1, 1, 512)], [torch.zeros(1, 1)])


@pytest.mark.parametrize("R,stride", [(64, 41216), (128, 82432)])
def test_page_layout(R, stride):
    a = synth.kv8_layout(R)
    assert a["page_stride"] == stride and stride % 128 == 0
    assert a["k_offset"] % 16 == 0 and a["scale_offset"] % 16 == 0
    assert a["kv_scale_offset"] == R * 512 and a["k_offset"] == R * 514
    assert a["scale_offset"] == a["k_offset"] + R * 128
