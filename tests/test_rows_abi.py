"""Struct layouts and refusals of the calls that rotate and prepare rows (no GPU:
every refusal returns before any CUDA call, and the pointers are fake)."""
import ctypes
import os
import subprocess

import pytest

from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20            # a fake, aligned address (never dereferenced)
INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 6


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return qli.lib()


@pytest.mark.parametrize("c_name,mirror", [
    ("qli_rotary", qli.RotaryArgs), ("qli_row_prep", qli.RowPrepArgs), ("qli_rotate_args", qli.RotateArgs),
    ("qli_prepare_args", qli.PrepareArgs), ("qli_append_args", qli.AppendArgs)])
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
    assert [getattr(mirror, f).offset for f in fields] == vals[1:]


def rotary(**over):
    a = qli.Rotary(64).args(0)
    for k, v in over.items():
        setattr(a, k, v)
    return a


ROTARY_REJECT = [(dict(layout=2), UNSUPPORTED), (dict(pairs=4), UNSUPPORTED), (dict(pairs=12), UNSUPPORTED),
                 (dict(pairs=72), UNSUPPORTED), (dict(pairs=-8), UNSUPPORTED), (dict(offset=4), UNSUPPORTED),
                 (dict(offset=-8), INVALID), (dict(offset=72), INVALID), (dict(magnitude=float("nan")), INVALID),
                 (dict(magnitude=float("inf")), INVALID), (dict(magnitude=1e300), INVALID)]


def good_rotate(**over):
    a = qli.RotateArgs(P, 8 * 128, 128, 4, 8, 128, 0, P, 2 * P, 8 * 128, 128)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,want", ROTARY_REJECT + [(dict(pairs=0), UNSUPPORTED)])
def test_rotate_refuses_rotations(L, over, want):
    assert L.qli_rotate(ctypes.byref(good_rotate()), ctypes.byref(rotary(**over)), None) == want


@pytest.mark.parametrize("over,want", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(D=132), UNSUPPORTED), (dict(D=8), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(positions=None), INVALID),
    (dict(x_stride_t=-8), INVALID), (dict(x=P + 8), ALIGNMENT), (dict(out=P + 8), ALIGNMENT),
    (dict(x_stride_h=132), ALIGNMENT), (dict(out_stride_t=1028), ALIGNMENT), (dict(positions=P + 2), ALIGNMENT),
    (dict(out_stride_h=64), INVALID), (dict(out_stride_t=512), INVALID),          # rows that overlap
    (dict(out_stride_t=128, out_stride_h=256), INVALID),
    (dict(out=P, out_stride_h=256, out_stride_t=2048), INVALID),                 # in place at other strides
    (dict(T=(1 << 27) + 1, out_stride_t=1024), UNSUPPORTED), (dict(D=65544), UNSUPPORTED)])
def test_rotate_refuses(L, over, want):
    assert L.qli_rotate(ctypes.byref(good_rotate(**over)), ctypes.byref(rotary()), None) == want


def test_rotate_refuses_no_arguments_and_undoing_nothing(L):
    assert L.qli_rotate(None, ctypes.byref(rotary()), None) == INVALID
    assert L.qli_rotate(ctypes.byref(good_rotate()), None, None) == INVALID
    zero = ctypes.byref(rotary(magnitude=0.0))
    assert L.qli_rotate(ctypes.byref(good_rotate(inverse=1)), zero, None) == INVALID
    assert L.qli_rotate(ctypes.byref(good_rotate(T=0, x=None, out=None, positions=None)), ctypes.byref(rotary()),
                        None) == qli.OK


def good_prep(width=128, **over):
    a = qli.RowPrepArgs(width, 1, 1e-6, 0, P, None, rotary())
    for k, v in over.items():
        setattr(a, k, v)
    return a


PREP_REJECT = [
    (dict(norm=3), UNSUPPORTED), (dict(norm=0), INVALID), (dict(bias=P), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(weight=P + 4), ALIGNMENT), (dict(norm=2, bias=P + 8), ALIGNMENT)]
PREP_REJECT += [(dict(rotary=rotary(**o)), w) for o, w in ROTARY_REJECT]


def good_prepare(**over):
    a = qli.PrepareArgs(P, 8 * 128, 128, 4, 8, P, 2 * P, 8 * 128, 128, P, qli.QUANT_INT8, 0)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,want", PREP_REJECT + [(dict(width=96), UNSUPPORTED), (dict(width=512), UNSUPPORTED)])
def test_prepare_refuses_preparations(L, over, want):
    assert L.qli_prepare_q(ctypes.byref(good_prepare()), ctypes.byref(good_prep(**over)), None) == want


@pytest.mark.parametrize("over,want", [
    (dict(quant_mode=3), UNSUPPORTED), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(x=None), INVALID),
    (dict(out=None), INVALID), (dict(positions=None), INVALID), (dict(scale_out=None), INVALID),
    (dict(out=P), INVALID), (dict(x=P + 2), ALIGNMENT), (dict(x_stride_t=1028), ALIGNMENT),
    (dict(out_stride_h=136), ALIGNMENT), (dict(quant_mode=0, out_stride_h=132), ALIGNMENT),
    (dict(out_stride_h=112), INVALID), (dict(positions=P + 2), ALIGNMENT), (dict(scale_out=P + 1), ALIGNMENT),
    (dict(quant_mode=0, out=P, out_stride_t=2048), INVALID)])
def test_prepare_refuses(L, over, want):
    assert L.qli_prepare_q(ctypes.byref(good_prepare(**over)), ctypes.byref(good_prep()), None) == want


def test_prepare_nothing_to_do(L):
    assert L.qli_prepare_q(ctypes.byref(good_prepare(T=0, x=None)), ctypes.byref(good_prep()), None) == qli.OK
    assert L.qli_prepare_q(None, ctypes.byref(good_prep()), None) == INVALID
    assert L.qli_prepare_q(ctypes.byref(good_prepare()), None, None) == INVALID


def good_append(**over):
    a = qli.AppendArgs(P, 512, P, 128, 4, P, P, P, 10, 82432, 128, 2, 2, 0, 0, 65536, 65792, 82176, None)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def _append(L, kv_prep=None, index_prep=None, **over):
    return L.qli_append_kv(ctypes.byref(good_append(**over)),
                           ctypes.byref(good_prep(512) if kv_prep is None else kv_prep),
                           ctypes.byref(good_prep() if index_prep is None else index_prep), None)


@pytest.mark.parametrize("over,want", [
    (dict(kv_mode=3), UNSUPPORTED), (dict(quant_mode=0), UNSUPPORTED), (dict(n=-1), INVALID),
    (dict(num_pages=-1), INVALID), (dict(n=(1 << 30) + 1), UNSUPPORTED), (dict(kv=None, index_k=None), INVALID),
    (dict(cache=None), INVALID), (dict(slot_mapping=None), INVALID), (dict(rows_per_page=32), UNSUPPORTED),
    (dict(page_stride=0), INVALID), (dict(kv_stride=504), INVALID), (dict(index_stride=120), INVALID),
    (dict(kv_stride=516), ALIGNMENT), (dict(index_stride=132), ALIGNMENT), (dict(kv=P + 8), ALIGNMENT),
    (dict(index_k=P + 8), ALIGNMENT), (dict(kv_offset=8), ALIGNMENT), (dict(k_offset=65800), ALIGNMENT),
    (dict(kv_scale_offset=65537), ALIGNMENT), (dict(scale_offset=82177), ALIGNMENT), (dict(kv_offset=-16), INVALID),
    (dict(scale_offset=82432 - 254), INVALID), (dict(k_offset=82432), INVALID), (dict(positions=None), INVALID),
    (dict(cache=P + 8), ALIGNMENT), (dict(page_stride=82440), ALIGNMENT), (dict(slot_mapping=P + 4), ALIGNMENT),
    (dict(positions=P + 2), ALIGNMENT), (dict(err_word=P + 2), ALIGNMENT),
    (dict(k_offset=65536), INVALID), (dict(scale_offset=65536), INVALID),        # parts that overlap
    (dict(kv_mode=0), INVALID), (dict(kv_scale_offset=1024), INVALID)])
def test_append_refuses(L, over, want):
    assert _append(L, **over) == want


@pytest.mark.parametrize("over,want", PREP_REJECT + [(dict(width=64), UNSUPPORTED)])
def test_append_refuses_preparations(L, over, want):
    if over.get("rotary") is None or over["rotary"].offset != 72:                 # 72 + 64 fit into 512
        assert _append(L, kv_prep=good_prep(**dict(dict(width=512), **over))) == want
    assert _append(L, index_prep=good_prep(**over)) == want


def test_append_nothing_to_do(L):
    assert _append(L, n=0, cache=None) == qli.OK
    assert L.qli_append_kv(None, None, None, None) == INVALID
    assert L.qli_append_kv(ctypes.byref(good_append()), None, ctypes.byref(good_prep()), None) == INVALID
    assert L.qli_append_kv(ctypes.byref(good_append()), ctypes.byref(good_prep(512)), None, None) == INVALID


# ---- the drafted trees ----------------------------------------------------------

def _tree(L, mask=P, words=1, **over):
    from test_kv_abi import good_attn
    return L.qli_kv_tree_attention(ctypes.byref(good_attn(False, **over)), mask, words, P, 1 << 40, None)


@pytest.mark.parametrize("kw,want", [
    (dict(mask=None), INVALID), (dict(mask=P + 4), ALIGNMENT), (dict(words=0), INVALID), (dict(words=-1), INVALID),
    (dict(words=257), UNSUPPORTED),
    (dict(indices=P, K=4), INVALID), (dict(ratio=2), UNSUPPORTED), (dict(residual=P), 4), (dict(window=-1), INVALID),
    (dict(k_lens=None), INVALID), (dict(D=576), UNSUPPORTED), (dict(q=P + 8), ALIGNMENT)])
def test_tree_refuses(L, kw, want):
    assert _tree(L, **kw) == want


def test_tree_nothing_to_do(L):
    assert _tree(L, mask=None, T=0) == qli.OK
    assert L.qli_kv_tree_attention(None, P, 1, None, 0, None) == INVALID
