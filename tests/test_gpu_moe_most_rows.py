"""The most rows that a plan takes, 2^30 of one choice each, grouped and brought back to their rows by the combination.

Exact: results are whole numbers under 2^8 and weights multiples of 1/4, by position and by row.  54 GB of device memory.
"""
import pytest
import torch

from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb
from test_gpu_moe import Plan
from test_gpu_mx import BF, DEV, stream

pytestmark = pytest.mark.gpu

ROWS, EXPERTS, D, SLICE = 1 << 30, 2, 8, 1 << 24


def by_place(first):
    p = torch.arange(first, first + SLICE, device=DEV)
    return ((p * 40503) >> 9).remainder_(251)[:, None] - torch.arange(D, device=DEV)


def by_row(rows):
    return (rows % 5 - 2) * 0.25


def test_most_rows_combined():
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("less than 80 GiB of free device memory")
    note("combination of 2^30 rows")
    ids = torch.empty(ROWS, dtype=torch.int32, device=DEV)
    weights = torch.empty(ROWS, device=DEV)
    y = torch.empty(ROWS, D, dtype=torch.bfloat16, device=DEV)
    order = torch.empty(ROWS, dtype=torch.int32, device=DEV)
    for r in range(0, ROWS, SLICE):
        rows = torch.arange(r, r + SLICE, device=DEV)
        ids[r:r + SLICE] = ((rows * 2654435761) >> 13) % 3 - 1
        weights[r:r + SLICE] = by_row(rows)
        y[r:r + SLICE] = by_place(r)
    out = torch.full((ROWS, D), 7.0, dtype=torch.bfloat16, device=DEV)
    with Plan(ROWS, EXPERTS, 1) as plan:
        lb.lora_moe_group(plan.at, ids.data_ptr(), ROWS, order.data_ptr(), 0, stream())
        lb.lora_moe_combine(plan.at, out.data_ptr(), D, y.data_ptr(), D, BF, weights.data_ptr(), 0, 0, BF, D, stream())
        torch.cuda.synchronize()
    last = -1
    for p in range(0, ROWS, SLICE):
        at = order[p:p + SLICE].long()
        key = ids[at].long()
        both = torch.where(key < 0, EXPERTS, key) * ROWS + at   # rises: the one stable order, every row once
        assert int(both[0]) > last and bool((both[1:] > both[:-1]).all()), f"positions from {p}"
        last = int(both[-1])
        want = (by_place(p) * by_row(at)[:, None] * (key >= 0)[:, None]).bfloat16()
        assert torch.equal(out[at], want), f"positions from {p}"
    del ids, weights, y, order, out
    torch.cuda.empty_cache()
