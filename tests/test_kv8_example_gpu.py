"""The decode-step example end to end on the GPU: writer, index-K writer, indexer,
both attention stages, merge and read-back, against attention computed on the
rows read back.

Bound: the rows read back are rounded to BF16 (2^-8 of |kv|, which is below 5 for
these normal values and moves a score of 512 terms by at most ~2^-8 * max|z| <
2^-5), each stage's output and the merged one by 2^-8 of values below 5."""
import importlib.util
import os

import pytest

from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    libbuild.build()
    qli.lib()
    spec = importlib.util.spec_from_file_location("kv8_decode", os.path.join(ROOT, "examples", "kv8_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("mode", [qli.QUANT_INT8, qli.QUANT_FP8], ids=["i8", "f8"])
def test_decode_steps(example, mode):
    pool = example.Pool([1, 700, 5000], 3, mode, seed=4)
    for i in range(3):
        step = example.decode_step(pool, topk=512, window=100)
        assert step["rows"].shape == (min(100, 2 + i), 512)
        assert example.check(pool, step) < 2.0 ** -4
    assert pool.lengths.tolist() == [4, 703, 5003]
    assert int(pool.err.item()) == 0


def test_command_line(example, capsys):
    example.main(["--requests", "3", "--context", "600", "--topk", "64", "--steps", "2", "--check"])
    assert capsys.readouterr().out.count("largest difference") == 2
