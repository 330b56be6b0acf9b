"""The largest batch that a plan takes, 2^26 rows of 16 choices: pairs and positions up to 2^30, and (in 4 bits, every pair
with an expert) more row tiles than one launch takes.

Everything is exact: logits and rows of X are among 256 patterns, whose choices and products come from a small batch or a
table, and sums are multiples of 2^-3 below 2^9.  70 GB of device memory.
"""
import numpy as np
import pytest
import torch

import mx_reference as R
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb
from test_gpu_moe import SOFTMAX, Plan
from test_gpu_mx import BF, DEV, F32, held, stream
from test_gpu_mx_experts import Experts

pytestmark = pytest.mark.gpu

ROWS, EXPERTS, TOP_K, PATTERNS, K = 1 << 26, 16, 16, 256, 8
PAIRS, SLICE = ROWS * TOP_K, 1 << 24


@pytest.fixture(scope="module")
def big():
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("less than 100 GiB of free device memory")
    pattern = ((torch.arange(ROWS, device=DEV) * 40503) >> 9).remainder_(PATTERNS).to(torch.uint8)
    with Plan(ROWS, EXPERTS, TOP_K) as plan:
        yield plan, pattern
    del pattern
    torch.cuda.empty_cache()


def spread(table, pattern):
    """table[pattern], in pieces that torch can index at once."""
    out = torch.empty(len(pattern), table.shape[1], dtype=table.dtype, device=DEV)
    for r in range(0, len(pattern), 1 << 20):
        out[r:r + (1 << 20)] = table[pattern[r:r + (1 << 20)].long()]
    return out


def check_order(order, offsets, ids):
    """Keys that do not fall and, among equal ones, pairs that rise: the one stable order."""
    count = torch.zeros(EXPERTS + 1, dtype=torch.int64, device=DEV)
    before = torch.tensor([-1], dtype=torch.int64, device=DEV)
    for p in range(0, PAIRS, SLICE):
        at = order[p:p + SLICE].long()
        assert int(at.min()) >= 0 and int(at.max()) < PAIRS
        key = ids.view(-1)[at].long()
        key = torch.where(key < 0, EXPERTS, key)
        count += torch.bincount(key, minlength=EXPERTS + 1)
        both = torch.cat([before, key * PAIRS + at])
        assert bool((both[1:] > both[:-1]).all()), f"positions from {p}"
        before = both[-1:]
    want = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), count.cumsum(0)])[:EXPERTS + 1]
    assert torch.equal(offsets.long(), want)


def test_largest_route(big):
    note("route of the largest batch")
    plan, pattern = big
    some = torch.randn(PATTERNS, EXPERTS, device=DEV, generator=torch.Generator(device=DEV).manual_seed(0)).bfloat16()

    def route(at, logits, rows, order, offsets):
        ids = torch.empty(rows, TOP_K, dtype=torch.int32, device=DEV)
        w = torch.empty(rows, TOP_K, device=DEV)
        lb.lora_moe_route(at, ids.data_ptr(), w.data_ptr(), order, offsets, logits.data_ptr(), EXPERTS, BF, rows, SOFTMAX, True, 1.0,
                          stream())
        return ids, w

    with Plan(PATTERNS, EXPERTS, TOP_K) as small:
        want_ids, want_w = route(small.at, some, PATTERNS, 0, 0)
    logits = spread(some, pattern)
    order = torch.empty(PAIRS, dtype=torch.int32, device=DEV)
    offsets = torch.empty(EXPERTS + 1, dtype=torch.int32, device=DEV)
    ids, w = route(plan.at, logits, ROWS, order.data_ptr(), offsets.data_ptr())
    for r in range(0, ROWS, SLICE):
        which = pattern[r:r + SLICE].long()
        assert torch.equal(ids[r:r + SLICE], want_ids[which]) and torch.equal(w[r:r + SLICE], want_w[which]), f"rows from {r}"
    check_order(order, offsets, ids)


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
def test_largest_group_product_and_combination(fmt, big):
    note(f"group, product and combination of the largest batch, format {fmt}")
    plan, pattern = big
    g = np.random.default_rng(0)
    dev = torch.Generator(device=DEV).manual_seed(1)
    one = np.full((EXPERTS, K, 1), 127, np.uint8)
    w = g.choice([-6.0, -3.0, -1.0, 0.0, 0.5, 1.0, 2.0, 4.0], (EXPERTS, K, K))
    packed = [(R.pack(R.codes_under(w[e], one[e], R.E2M1), R.E2M1), R.pad_scales(one[e], K)) for e in range(EXPERTS)]
    bits = (np.arange(PATTERNS)[:, None] >> np.arange(K)) & 1
    table = torch.from_numpy(np.einsum("pk,eok->epo", bits, w).astype(np.float32)).to(DEV).reshape(EXPERTS * PATTERNS, K)
    ones = np.full((PATTERNS, 1), 127, np.uint8)
    xq = spread(torch.from_numpy(R.pack(R.codes_under(bits.astype(float), ones, fmt), fmt)).to(DEV), pattern)
    xs = spread(torch.from_numpy(R.pad_scales(ones, K)).to(DEV), pattern)
    ids = torch.randint(-1 if fmt == R.E4M3 else 0, EXPERTS, (ROWS, TOP_K), dtype=torch.int32, device=DEV, generator=dev)
    order = torch.empty(PAIRS, dtype=torch.int32, device=DEV)
    offsets = torch.empty(EXPERTS + 1, dtype=torch.int32, device=DEV)
    lb.lora_moe_group(plan.at, ids.data_ptr(), ROWS, order.data_ptr(), offsets.data_ptr(), stream())
    check_order(order, offsets, ids)

    y = torch.full((PAIRS, K), 7.0, device=DEV)
    with Experts(packed, K, K, False) as x:
        lb.lora_mx_expert_linear(x.at, plan.at, y.data_ptr(), K, 0, 0, 0, 0, F32, *held(xq, xs), fmt, lb.LORA_MOE_ROWS, 0,
                                 lb.LORA_ACT_NONE, stream())
    for p in range(0, PAIRS, SLICE):
        at = order[p:p + SLICE].long()
        e = ids.view(-1)[at].long()
        want = table[(e.clamp(min=0) * PATTERNS + pattern[at >> 4].long())]
        want[e < 0] = 7.0
        assert torch.equal(y[p:p + SLICE], want), f"positions from {p}"

    weights = torch.randint(-2, 3, (ROWS, TOP_K), device=DEV, generator=dev, dtype=torch.int32).float() * 0.25
    out = torch.empty(ROWS, K, device=DEV)
    lb.lora_moe_combine(plan.at, out.data_ptr(), K, y.data_ptr(), K, F32, weights.data_ptr(), 0, 0, F32, K, stream())
    for r in range(0, ROWS, SLICE // TOP_K):
        e = ids[r:r + SLICE // TOP_K].long()
        v = table[e.clamp(min=0) * PATTERNS + pattern[r:r + SLICE // TOP_K].long()[:, None]]
        want = (v * (weights[r:r + SLICE // TOP_K] * (e >= 0))[:, :, None]).sum(1)
        assert torch.equal(out[r:r + SLICE // TOP_K], want), f"rows from {r}"
