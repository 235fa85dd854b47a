"""Block tables that are slices of wider ones, or whose only row has any stride:
positions past the slice are skipped and flagged although the columns beside it
name pages of the pool, and a table of one row is as wide as it is."""
import pytest

from kv8_cases import KVCase
from oracle import kv8
from test_kv_attn_gpu import _lib, compare, run  # noqa: F401

pytestmark = pytest.mark.gpu

PAGE, KLEN = 8, 2                  # error bits: a page or position, a request's length


def _beside(case):
    """The case's table between columns that name page 0."""
    import torch
    n = case.bt.shape[1]
    wide = torch.zeros(case.B + 1, n + 9, dtype=torch.int32, device="cuda")
    wide[:case.B, 3:3 + n] = torch.from_numpy(case.bt).cuda()
    return wide[:case.B, 3:3 + n]


@pytest.mark.parametrize("quant", [kv8.INT8, kv8.FP8], ids=["i8", "f8"])
def test_listed_positions_past_a_slice(quant):
    case = KVCase(141, [900, 700], [1, 2], 1, 64, quant, K=200)
    cap = case.bt.shape[1] * case.R
    bad = {(0, 7): cap, (0, 8): cap + 5 * case.R, (1, 0): cap + 1, (2, 199): cap + 9 * case.R}
    for (t, k), j in bad.items():
        case.indices[t, 0, k] = j
    got = run(case, err_want=PAGE, block_table=_beside(case))
    for t, k in bad:
        case.indices[t, 0, k] = -1
    compare(case, got)


def test_visible_positions_past_a_slice():
    import torch
    case = KVCase(142, [512, 400], [1, 1], 1, 64, kv8.FP8)
    cap = case.bt.shape[1] * case.R
    assert cap == 512
    k = torch.tensor([cap + 1, 400], dtype=torch.int32, device="cuda")
    compare(case, run(case, err_want=KLEN, k_lens=k, block_table=_beside(case)))


@pytest.mark.parametrize("listed", [False, True], ids=["dense", "listed"])
def test_a_row_of_any_stride(listed):
    import torch
    case = KVCase(143, [1000], [2], 1, 32, kv8.INT8, K=300 if listed else None)
    bt = torch.from_numpy(case.bt).cuda().as_strided((1, 8), (1, 1))
    compare(case, run(case, block_table=bt))


def test_a_table_of_one_column():
    import torch
    case = KVCase(144, [100, 128, 5], [1, 1, 1], 1, 48, kv8.FP8)
    bt = torch.from_numpy(case.bt).cuda().as_strided((3, 1), (1, 3))
    compare(case, run(case, block_table=bt))
