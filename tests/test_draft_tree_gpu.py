"""The calls of a drafted token tree together, as examples/kv8_draft_tree.py makes
them: rows and queries against the float64 oracle, attention against attention over
the rows read back, the accepted path against a pool that never held the tree."""
import os
import sys

import numpy as np
import pytest

from oracle import kv8
from oracle import rows as oracle
from sparse_attention_indexer_qli_gb300 import build as libbuild
from sparse_attention_indexer_qli_gb300 import qli

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    qli.lib()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
def test_verify_step(quant, heads):
    import torch

    import kv8_draft_tree as ex
    r = ex.Requests([1, 100, 1500, 3000], 24, quant, seed=3)
    step = ex.verify_step(r, ex.TREE, heads, topk=256)
    torch.cuda.synchronize()
    assert int(r.err.item()) == 0
    # merged: two stages of 2^-11 of the largest value each and three roundings to BF16 of
    # 2^-8 (both stages and the merge), over rows whose values are below 8
    rows = qli.read_kv(r.cache, torch.arange(r.cache.shape[0] * r.R, device="cuda"), **r.kv_geometry())
    top = float(rows.abs().max())
    assert ex.check(r, step) <= top * (2 * 2.0 ** -11 + 3 * 2.0 ** -8)
    # the queries, and the output rotated back
    pos, R = step["position"].cpu().numpy(), r.layer.rotary
    x = oracle.normalise(f64(step["x"]), "rms", r.layer.queries.weight.double().cpu().numpy())
    want = oracle.rotate(x, pos, R.frequencies, ex.D - ex.ROT, False)
    assert np.all(np.abs(f64(step["q"]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -16 * np.abs(want).max())
    m = f64(step["merged"])
    want = oracle.rotate(m, pos, R.frequencies, ex.D - ex.ROT, False, inverse=True)
    assert np.all(np.abs(f64(step["out"]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -16 * np.abs(m).max())


def test_the_accepted_path_leaves_what_plain_decoding_would():
    import torch

    import kv8_draft_tree as ex
    r = ex.Requests([300, 77], 24, kv8.FP8, seed=5)
    step = ex.verify_step(r, ex.TREE, 64, topk=64)
    path = [0, 1, 3, 6]
    ex.accept(r, step, path)
    assert r.lengths.tolist() == [304, 81]
    want = ex.Requests([300, 77], 24, kv8.FP8, seed=5)
    n = len(ex.TREE)
    for b in range(2):
        for depth, i in enumerate(path):
            t, at = b * n + i, torch.tensor([int(want.lengths[b]) + depth], device="cuda")
            want.append(torch.tensor([b], device="cuda"), at, at, step["kv"][t:t + 1], step["index_k"][t:t + 1])
    for b, length in enumerate([304, 81]):
        place = torch.arange(length, device="cuda")
        slots = r.block_table[b, place // r.R].long() * r.R + place % r.R
        page, row, L = slots // r.R, slots % r.R, r.layout
        for off, width in ((L["kv_offset"], 512), (L["kv_scale_offset"], 2), (L["k_offset"], 128), (L["scale_offset"], 2)):
            cols = off + row[:, None] * width + torch.arange(width, device="cuda")
            assert torch.equal(r.cache[page[:, None], cols], want.cache[page[:, None], cols])


def test_the_example_runs(capsys):
    import kv8_draft_tree as ex
    ex.main(["--requests", "3", "--context", "700", "--steps", "3", "--check", "--quant", "int8", "--heads", "32"])
    lines = capsys.readouterr().out.strip().splitlines()
    assert len(lines) == 3 and all("largest difference" in line for line in lines)
