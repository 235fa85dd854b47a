"""The plans of rotations and row preparations, and the binding of their calls (on
the CPU, see fake_cuda): frequencies, refusals, devices and streams."""
import ctypes
import math

import numpy as np
import pytest
import torch

from fake_cuda import DEVICE, GEOMETRY, FakeStream, attention_inputs, fake, on_gpu  # noqa: F401
from oracle import rows as oracle
from sparse_attention_indexer_qli_gb300 import qli


@pytest.mark.parametrize("dim", [16, 64, 128])
@pytest.mark.parametrize("kw", [{}, dict(base=500000.0), dict(factor=4.0), dict(factor=16.0, trained=8192),
                                dict(factor=40.0, trained=4096, ramp=(2.0, 20.0))])
def test_frequencies(dim, kw):
    r = qli.Rotary(dim, **kw)
    want = oracle.frequencies(dim, **kw)
    np.testing.assert_allclose(r.frequencies, want, rtol=1e-14)
    # turns in 2^-64: off by half a unit and by what FP64 is
    got = np.array([t / 2.0 ** 64 for t in r.args(0).turns[:dim // 2]])
    np.testing.assert_allclose(got, want / (2 * math.pi), rtol=4e-16, atol=2.0 ** -64)
    assert not any(r.args(0).turns[dim // 2:])


def test_angles_of_far_positions_are_exact():
    """The whole-number product modulo 2^64 is the fraction of a turn; an FP64
    product of position and frequency is off by less than 1e-7 of one here."""
    r = qli.Rotary(64)
    for p in (0, 1, -1, 12345, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
        for t, f in zip(r.args(0).turns[:32], r.frequencies):
            got = (p * t) % 2 ** 64 / 2.0 ** 64
            want = p * f / (2 * math.pi)
            assert abs((got - want + 0.5) % 1.0 - 0.5) < 1e-6


def test_frequencies_of_ones_own():
    r = qli.Rotary(16, frequencies=[0.0, 1.0, -1.0, math.pi, 7.0, 2 * math.pi, 1e-9, 0.5])
    half = 1 << 63
    assert r.args(0).turns[0] == 0 and r.args(0).turns[3] == half
    assert (r.args(0).turns[1] + r.args(0).turns[2]) % 2 ** 64 == 0
    assert r.args(0).turns[5] in (0, 1, 2 ** 64 - 1)              # a whole turn


@pytest.mark.parametrize("kw", [dict(dim=8), dict(dim=24), dict(dim=144), dict(layout="pairs"), dict(magnitude=0.0),
                                dict(magnitude=float("nan")), dict(base=0.0), dict(factor=0.0), dict(factor=float("inf")),
                                dict(trained=0), dict(trained=8, ramp=(2.0, 1.0)), dict(frequencies=[1.0]),
                                dict(frequencies=[float("inf")] * 32)])
def test_rotary_refuses(kw):
    with pytest.raises(ValueError):
        qli.Rotary(**dict(dict(dim=64), **kw))


def w(n, elsewhere=False, dtype=torch.float32):
    return on_gpu(torch.ones(n, dtype=dtype), elsewhere)


@pytest.mark.parametrize("kw,error", [
    (dict(norm="batch"), ValueError), (dict(weight=w(128)), ValueError), (dict(norm="rms", bias=w(128)), ValueError),
    (dict(norm="rms", weight=w(64)), ValueError), (dict(norm="rms", weight=torch.ones(128)), TypeError),
    (dict(norm="rms", weight=w(128, dtype=torch.bfloat16)), TypeError),
    (dict(norm="rms", weight=on_gpu(torch.ones(256))[::2]), ValueError),
    (dict(norm="layer", weight=w(128), bias=w(128, True)), ValueError)])
def test_row_prep_refuses(kw, error):
    with pytest.raises(error):
        qli.RowPrep(128, **kw)


def test_row_prep_packs():
    weight, bias = w(128), w(128)
    p = qli.RowPrepArgs.from_buffer_copy(
        qli.RowPrep(128, norm="layer", weight=weight, bias=bias, eps=0.5, rotary=qli.Rotary(32, layout="half"),
                    offset=96).packed)
    assert (p.width, p.norm, p.eps, p.weight, p.bias) == (128, 2, 0.5, weight.data_ptr(), bias.data_ptr())
    assert (p.rotary.pairs, p.rotary.layout, p.rotary.offset, p.rotary.magnitude) == (16, 1, 96, 1.0)
    p = qli.RowPrepArgs.from_buffer_copy(qli.RowPrep(512).packed)
    assert (p.norm, p.weight, p.rotary.pairs) == (0, None, 0)


@pytest.fixture
def lib(fake):  # noqa: F811
    """The fake library with the calls of this file."""
    f = fake.lib

    def note(name, mirror):
        def call(a, *rest):
            return f._note(name, mirror.from_buffer_copy(a), *rest)
        return call
    f.qli_rotate = note("rotate", qli.RotateArgs)
    f.qli_prepare_q = note("prepare_q", qli.PrepareArgs)
    f.qli_append_kv = note("append_kv", qli.AppendArgs)
    f.qli_kv_tree_attention = note("kv_tree_attention", qli.KVAttnArgs)
    return fake


def bf16(*shape):
    return on_gpu(torch.zeros(*shape, dtype=torch.bfloat16))


def i32(*shape):
    return on_gpu(torch.zeros(*shape, dtype=torch.int32))


def i64(*shape):
    return on_gpu(torch.zeros(*shape, dtype=torch.int64))


ROT = qli.Rotary(64)
PAGES = dict(rows_per_page=64, page_stride=41216, kv_offset=0, kv_scale_offset=32768, k_offset=32896,
             scale_offset=41088)


def _rotate():
    return (lambda x, positions, **kw: qli.rotate(x, positions, ROT, offset=64, **kw)), \
        dict(x=bf16(3, 2, 128), positions=i32(3), out=bf16(3, 2, 128))


def _prepare():
    prep = qli.RowPrep(128, rotary=ROT)
    return (lambda x, positions, **kw: qli.prepare_q(x, positions, prep, quant_mode=qli.QUANT_FP8, **kw)), \
        dict(x=bf16(3, 2, 128), positions=i32(3), out=on_gpu(torch.zeros(3, 2, 128, dtype=torch.int8)),
             scale_out=on_gpu(torch.zeros(3, 2, dtype=torch.int16)))


def _append():
    kv, index = qli.RowPrep(512, rotary=ROT, offset=448), qli.RowPrep(128, norm="layer")
    return (lambda **kw: qli.append_kv(kv_prep=kv, index_prep=index, **PAGES, **kw)), \
        dict(kv=bf16(3, 512), index_k=bf16(3, 128), positions=i32(3), slot_mapping=i64(3),
             cache=on_gpu(torch.zeros(2, 41216, dtype=torch.uint8)), err_word=i32(1))


def _tree():
    kw = attention_inputs()
    kw.pop("indices")
    kw.update(k_lens=i32(2), tree_mask=i64(3, 2), out=bf16(3, 2, 512), lse=on_gpu(torch.zeros(3, 2)),
              workspace=on_gpu(torch.zeros(4096, dtype=torch.uint8)), err_word=i32(1))
    return qli.kv_tree_attention, kw


CALLS = [_rotate, _prepare, _append, _tree]
IDS = ["rotate", "prepare", "append", "tree"]


@pytest.mark.parametrize("make", CALLS, ids=IDS)
def test_a_tensor_of_another_device_is_refused(lib, make):
    call, kw = make()
    call(**kw)
    assert len(lib.lib.calls) == 1
    for name in [n for n, v in kw.items() if isinstance(v, torch.Tensor)]:
        with pytest.raises(ValueError, match="device"):
            call(**dict(kw, **{name: on_gpu(kw[name], elsewhere=True)}))
        with pytest.raises(TypeError):
            call(**dict(kw, **{name: torch.zeros(kw[name].shape, dtype=kw[name].dtype)}))
        with pytest.raises(TypeError):
            call(**dict(kw, **{name: on_gpu(torch.zeros(kw[name].shape, dtype=torch.float64))}))
    assert len(lib.lib.calls) == 1


@pytest.mark.parametrize("make", CALLS, ids=IDS)
def test_a_device_that_is_not_current_is_refused(lib, make):
    call, kw = make()
    there = {n: on_gpu(v, elsewhere=True) if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    with pytest.raises(ValueError, match="current device"):
        call(**there)
    lib.device = DEVICE + 1
    call(**there)
    assert len(lib.lib.calls) == 1


@pytest.mark.parametrize("make", CALLS, ids=IDS)
def test_refusals_of_the_library_raise(lib, make):
    call, kw = make()
    lib.lib.status = 2
    with pytest.raises(qli.QLIError, match="unsupported"):
        call(**kw)


@pytest.mark.parametrize("make,outputs", [(_rotate, ["out"]), (_prepare, ["out", "scale_out"]),
                                          (_tree, ["out", "lse"])], ids=["rotate", "prepare", "tree"])
def test_another_stream_gets_its_own_memory(lib, make, outputs):
    call, kw = make()
    for name in outputs + ["workspace"]:
        kw.pop(name, None)
    here, there = FakeStream("here", 11), FakeStream("there", 12)
    with lib.on(here):
        results = call(stream=there, **kw)
    assert lib.lib.calls[-1][1][-1] == 12
    results = results if isinstance(results, tuple) else (results,)
    assert len(lib.made) >= len(outputs) and all(s is there for s, _ in lib.made)
    assert set(lib.recorded) == {(t.data_ptr(), here) for t in results}


def test_weights_of_another_device_are_refused(lib):
    prep = qli.RowPrep(128, norm="rms", weight=w(128, elsewhere=True))
    with pytest.raises(ValueError, match="weights"):
        qli.prepare_q(bf16(3, 2, 128), None, prep)
    with pytest.raises(ValueError, match="weights"):
        qli.append_kv(None, bf16(3, 128), None, i64(3), on_gpu(torch.zeros(2, 41216, dtype=torch.uint8)),
                      index_prep=prep, **PAGES)
    assert not lib.lib.calls


def test_strides_of_one_token_or_head_may_be_any(lib):
    x = on_gpu(torch.zeros(1, 2, 128, dtype=torch.bfloat16).as_strided((1, 2, 128), (3, 128, 1)))
    qli.rotate(x, i32(1), ROT, out=x)
    a = lib.lib.calls[-1][1][0]
    assert (a.x_stride_t, a.x_stride_h) == (a.out_stride_t, a.out_stride_h) == (256, 128)
    x = on_gpu(torch.zeros(5 * 136, dtype=torch.bfloat16).as_strided((5, 1, 128), (136, 1, 1)))
    qli.rotate(x, i32(5), ROT)
    a = lib.lib.calls[-1][1][0]
    assert (a.x_stride_t, a.x_stride_h, a.out_stride_t, a.out_stride_h) == (136, 128, 128, 128)


@pytest.mark.parametrize("call", [
    lambda: qli.rotate(bf16(3, 128), i32(3), ROT), lambda: qli.rotate(bf16(3, 128, 2).transpose(1, 2), i32(3), ROT),
    lambda: qli.rotate(bf16(3, 2, 128), i32(2), ROT), lambda: qli.rotate(bf16(3, 2, 128), i32(6)[::2], ROT),
    lambda: qli.rotate(bf16(3, 2, 128), i32(3), ROT, out=bf16(3, 2, 64)),
    lambda: qli.prepare_q(bf16(3, 2, 64), None, qli.RowPrep(128)),
    lambda: qli.prepare_q(bf16(3, 2, 128), None, qli.RowPrep(128, rotary=ROT)),
    lambda: qli.prepare_q(bf16(3, 2, 128), None, qli.RowPrep(128), quant_mode=0),
    lambda: qli.prepare_q(bf16(3, 2, 128), None, qli.RowPrep(128), scale_out=on_gpu(torch.zeros(3, 2, dtype=torch.int16))),
    lambda: qli.append_kv(bf16(3, 512), None, None, i64(2), on_gpu(torch.zeros(2, 41216, dtype=torch.uint8)),
                          kv_prep=qli.RowPrep(512), **PAGES),
    lambda: qli.append_kv(bf16(3, 512), None, None, i64(3), on_gpu(torch.zeros(2, 41216, dtype=torch.uint8)), **PAGES),
    lambda: qli.append_kv(bf16(3, 512), None, None, i64(3), on_gpu(torch.zeros(2, 41216, dtype=torch.uint8)),
                          kv_prep=qli.RowPrep(128), **PAGES),
    lambda: qli.append_kv(bf16(3, 512), None, None, i64(3), on_gpu(torch.zeros(2, 41216, dtype=torch.uint8)),
                          kv_prep=qli.RowPrep(512, rotary=ROT), **PAGES),
    lambda: qli.append_kv(bf16(3, 256), None, None, i64(3), on_gpu(torch.zeros(2, 41216, dtype=torch.uint8)),
                          kv_prep=qli.RowPrep(512), **PAGES)])
def test_shapes_are_refused(lib, call):
    with pytest.raises(ValueError):
        call()
    assert not lib.lib.calls


@pytest.mark.parametrize("mask,words", [((3,), 1), ((3, 1), 1), ((3, 4), 4)])
def test_tree_masks(lib, mask, words):
    call, kw = _tree()
    kw["tree_mask"] = i64(*mask)
    call(**kw)
    name, (a, m, n, ws, size, stream) = lib.lib.calls[-1]
    assert name == "kv_tree_attention" and m == kw["tree_mask"].data_ptr() and n == words
    assert (a.ratio, a.indices, a.residual) == (1, None, None)


@pytest.mark.parametrize("over", [dict(tree_mask=i64(4, 1)), dict(tree_mask=i64(3, 0)), dict(tree_mask=i64(3, 2, 1)),
                                  dict(tree_mask=i64(3, 4)[:, ::2]), dict(k_lens=None), dict(k_lens=i32(3))])
def test_tree_arguments_are_refused(lib, over):
    call, kw = _tree()
    with pytest.raises(ValueError):
        call(**dict(kw, **over))
    assert not lib.lib.calls


def test_none_as_a_tree_mask_is_refused(lib):
    call, kw = _tree()
    with pytest.raises(TypeError):
        call(**dict(kw, tree_mask=None))


def test_the_whole_number_of_bytes():
    assert ctypes.sizeof(qli.RotaryArgs) == len(ROT.packed(0)) == 536
