"""The frequencies of extended contexts: which blend `qli.Rotary` makes, and how another
one is passed (no GPU)."""
import math
import os

import numpy as np

from oracle import rows as oracle
from sparse_attention_indexer_qli_gb300 import qli

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_blend_is_linear_in_the_turns():
    r = qli.Rotary(64, factor=16.0, trained=8192)
    for i, f in enumerate(r.frequencies):
        plain = 10000.0 ** (-i / 32)
        turns = 8192 * plain / (2 * math.pi)
        stays = min(1.0, max(0.0, (turns - 1) / 31))
        assert math.isclose(f, plain * stays + plain / 16 * (1 - stays), rel_tol=1e-14)
    assert np.allclose(r.frequencies, oracle.frequencies(64, factor=16.0, trained=8192), rtol=1e-14, atol=0)


def test_the_other_blend_as_the_readme_passes_it():
    """Linear in the pair's number: the plan has those frequencies, and they are not its own."""
    lines = open(os.path.join(ROOT, "README.md")).read().split("pair = lambda turns", 1)[1].split("```")[0]
    names = {"math": math, "qli": qli}
    exec("pair = lambda turns" + lines, names)
    r, i = names["rotary"], np.arange(32)
    assert (names["low"], names["high"]) == (12, 25)
    plain = 10000.0 ** (-i / 32)
    want = np.where(i <= 12, plain, np.where(i >= 25, plain / 16, plain + (plain / 16 - plain) * (i - 12) / 13))
    assert np.allclose(r.frequencies, want, rtol=1e-14, atol=0)
    assert r._turns == [round(f / (2 * math.pi) * 2 ** 64) for f in r.frequencies]
    own = np.asarray(qli.Rotary(64, factor=16.0, trained=8192).frequencies)
    ratio = np.asarray(r.frequencies) / own
    assert np.flatnonzero(np.abs(ratio - 1) > 1e-12).tolist() == list(range(13, 25))
    assert 2.7 < ratio.max() < 2.8 and ratio.min() < 1
