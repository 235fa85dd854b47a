"""Pins of the 8-bit KV oracle (oracle/kv8.py): codes against brute force over
the whole grid, known rows, the attention against a plain double loop and its
invariants, the merge against attention over the union."""
import numpy as np
import pytest

from oracle import kv8


def test_e4m3_grid_and_rounding():
    v = kv8.e4m3_values()
    assert v[0x7E] == 448.0 and v[1] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0x38] == 1.0
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF]) and v[0xBC] == -1.5
    finite = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    assert np.array_equal(kv8.e4m3_codes(v[finite]), finite)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(500) * 10.0 ** rng.integers(-4, 4, 500),
                        (v[:126] + v[1:127]) / 2, [449.0, 1e9]])     # every tie
    got = v[kv8.e4m3_codes(x)]
    grid = v[finite]
    for xi, gi in zip(x, got):
        d = np.abs(grid - np.clip(xi, -448, 448))
        assert abs(gi - np.clip(xi, -448, 448)) == d.min()
    ties = kv8.e4m3_codes((v[:126] + v[1:127]) / 2)
    assert np.all(ties % 2 == 0)


def test_bf16_rounding_matches_torch():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(1).standard_normal(4000).astype(np.float32)
    want = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    assert np.array_equal(kv8.f32_to_bf16(x), want)


def test_known_rows():
    x = np.zeros((4, 512), dtype=np.float32)
    x[1, 3] = 127.0
    x[1, 4] = -2.5              # a tie under scale 1: even
    x[2, :] = 2.0 ** -40        # scale rounds to zero
    x[3, 0] = 3.0e38            # scale capped at 65504
    bits = kv8.f32_to_bf16(x)
    c, s = kv8.quantise_rows(bits, kv8.INT8)
    s = s.view(np.float16)
    assert s[0] == 0 and not c[0].any()
    assert s[1] == 1 and c[1].view(np.int8)[3] == 127 and c[1].view(np.int8)[4] == -2
    assert s[2] == 0 and not c[2].any()
    assert s[3] == 65504 and c[3].view(np.int8)[0] == 127
    c, s = kv8.quantise_rows(bits, kv8.FP8)
    assert not c[0].any() and not c[2].any() and c[3][0] == 0x7E


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8])
def test_quantisation_error_is_half_a_step(quant):
    rng = np.random.default_rng(2)
    bits = kv8.f32_to_bf16(rng.standard_normal((50, 512)))
    x = kv8.bf16_to_f64(bits)
    y = kv8.rows(*kv8.quantise_rows(bits, quant), quant)
    amax = np.abs(x).max(axis=1, keepdims=True)
    if quant == kv8.INT8:
        assert np.all(np.abs(x - y) <= 0.5 * amax / 127 * (1 + 2.0 ** -9) + 127 * amax / 127 * 2.0 ** -11)
    else:
        assert np.all(np.abs(x - y) <= np.abs(x) * 2.0 ** -4 + amax / 448 * 2.0 ** -9 + np.abs(x) * 2.0 ** -10)


def test_visible_counts():
    # 10 raw tokens at ratio 2, the last 3 are queries: 8, 9 and 10 tokens seen
    assert [kv8.visible(3, i, 5, 0, 2) for i in range(3)] == [4, 4, 5]
    assert [kv8.visible(3, i, 5, 1, 2) for i in range(3)] == [4, 5, 5]
    assert [kv8.visible(4, i, 4, 0, 1) for i in range(4)] == [1, 2, 3, 4]
    assert kv8.visible(5, 0, 1, 0, 2) == 0


def test_attention_against_a_plain_loop():
    rng = np.random.default_rng(3)
    q, kv = rng.standard_normal((3, 8)), rng.standard_normal((5, 8))
    o, lse = kv8.attend(q, kv, 0.7)
    for h in range(3):
        e = [np.exp(0.7 * sum(q[h, d] * kv[j, d] for d in range(8))) for j in range(5)]
        assert abs(lse[h] - np.log(sum(e))) < 1e-12
        for d in range(8):
            assert abs(o[h, d] - sum(e[j] * kv[j, d] for j in range(5)) / sum(e)) < 1e-12
    o, lse = kv8.attend(q, kv[:0], 0.7)
    assert not o.any() and np.all(np.isneginf(lse))


def test_merge_is_attention_over_the_union():
    rng = np.random.default_rng(4)
    q, kv = rng.standard_normal((3, 16)), rng.standard_normal((20, 16))
    o, lse = kv8.attend(q, kv, 0.5)
    parts = [kv8.attend(q, kv[a:b], 0.5) for a, b in ((0, 3), (3, 3), (3, 11), (11, 20))]
    got, got_lse = kv8.merge([p[0][None] for p in parts], [p[1][None] for p in parts])
    assert np.allclose(got[0], o, atol=1e-12) and np.allclose(got_lse[0], lse, atol=1e-12)
    none = kv8.merge([parts[1][0][None]] * 2, [parts[1][1][None]] * 2)
    assert not none[0].any() and np.all(np.isneginf(none[1]))
