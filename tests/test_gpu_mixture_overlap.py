"""Mixture layers' calls beside each other: products that share weights or a plan on streams of their own, batches of two
plans on two streams, and two captured batches that take turns with one plan.  The bits are those of the calls one by one."""
import numpy as np
import pytest
import torch

import mx_reference as R
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb
from test_gpu_moe import SOFTMAX, Plan, logits
from test_gpu_mx import BF, DEV, F32, held, rand, stream
from test_gpu_mx_experts import Experts

pytestmark = pytest.mark.gpu

EXPERTS, TOP_K, K, F = 6, 2, 520, 264


class Batch:
    """Router, gated product into blocks, product back, combination, on buffers of its own."""

    def __init__(self, rows, seed, plan, up, down):
        self.rows, self.plan, self.up, self.down = rows, plan, up, down
        self.logits = logits(seed, rows, EXPERTS, BF)[0]
        self.xq, self.xs = (torch.from_numpy(t).to(DEV) for t in R.quantize(rand(seed, rows, K, 0.3), R.E4M3))
        self.ids = torch.empty(rows, TOP_K, dtype=torch.int32, device=DEV)
        self.w = torch.empty(rows, TOP_K, device=DEV)
        self.aq = torch.zeros(rows * TOP_K, lb.lora_mx_code_bytes(F, R.E4M3), dtype=torch.uint8, device=DEV)
        self.a_s = torch.zeros(rows * TOP_K, lb.lora_mx_scale_bytes(F), dtype=torch.uint8, device=DEV)
        self.y = torch.zeros(rows * TOP_K, K, device=DEV)
        self.out = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)

    def route(self):
        lb.lora_moe_route(self.plan.at, self.ids.data_ptr(), self.w.data_ptr(), 0, 0, self.logits.data_ptr(), EXPERTS, BF, self.rows,
                          SOFTMAX, True, 1.0, stream())

    def up_product(self):
        lb.lora_mx_expert_linear(self.up.at, self.plan.at, 0, 0, *held(self.aq, self.a_s), BF, *held(self.xq, self.xs), R.E4M3,
                                 lb.LORA_MOE_ROWS, 0, lb.LORA_ACT_SWIGLU, stream())

    def down_product(self):
        lb.lora_mx_expert_linear(self.down.at, self.plan.at, self.y.data_ptr(), K, 0, 0, 0, 0, F32, *held(self.aq, self.a_s), R.E4M3,
                                 lb.LORA_MOE_PAIRS, 0, lb.LORA_ACT_NONE, stream())

    def combine(self):
        lb.lora_moe_combine(self.plan.at, self.out.data_ptr(), K, self.y.data_ptr(), K, F32, self.w.data_ptr(), 0, 0, BF, K, stream())

    def step(self):
        self.route()
        self.up_product()
        self.down_product()
        self.combine()

    def clear(self):
        for t in (self.aq, self.a_s, self.y, self.out):
            t.zero_()

    def results(self):
        return [t.clone() for t in (self.ids, self.w, self.aq, self.a_s, self.y, self.out)]


@pytest.fixture(scope="module")
def weights():
    g = np.random.default_rng(0)
    up = [R.quantize(g.standard_normal((2 * F, K)) * K ** -0.5, R.E2M1) for _ in range(EXPERTS)]
    down = [R.quantize(g.standard_normal((K, F)) * F ** -0.5, R.E2M1) for _ in range(EXPERTS)]
    with Experts(up, 2 * F, K, True) as u, Experts(down, K, F, False) as d:
        yield u, d


def same(got, want, what):
    assert all(torch.equal(a, b) for a, b in zip(got, want)), what


@pytest.mark.parametrize("rows", [(30, 41), (900, 1300)])
def test_two_batches_on_two_streams(rows, weights):
    note(f"two batches on two streams, {rows} rows")
    with Plan(rows[0], EXPERTS, TOP_K) as p, Plan(rows[1], EXPERTS, TOP_K) as q:
        batches = [Batch(rows[0], 1, p, *weights), Batch(rows[1], 2, q, *weights)]
        want = []
        for b in batches:
            b.step()
            torch.cuda.synchronize()
            want.append(b.results())
            b.clear()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(4):
            for s, b in zip(streams, batches):
                with torch.cuda.stream(s):
                    b.step()
        torch.cuda.synchronize()
        for b, w in zip(batches, want):
            same(b.results(), w, f"{b.rows} rows")


def test_products_of_one_plan_on_two_streams(weights):
    rows = 700
    note("products of one plan on two streams")
    with Plan(rows, EXPERTS, TOP_K) as plan:
        a = Batch(rows, 3, plan, *weights)
        b = Batch(rows, 4, plan, *weights)
        want = []
        a.route()
        for x in (a, b):     # b's rows under a's choices
            x.up_product()
            x.down_product()
            torch.cuda.synchronize()
            want.append([x.aq.clone(), x.a_s.clone(), x.y.clone()])
            x.clear()
        torch.cuda.synchronize()
        for s, x in ((torch.cuda.Stream(), a), (torch.cuda.Stream(), b)):
            with torch.cuda.stream(s):
                x.up_product()
                x.down_product()
        torch.cuda.synchronize()
        for x, w in zip((a, b), want):
            same([x.aq, x.a_s, x.y], w, "one plan")


def test_two_captured_batches_of_one_plan(weights):
    """Each graph makes its own grouping: replayed in any order, with an eager batch of the same plan between."""
    sizes = (900, 20, 300)
    note("two captured batches of one plan")
    with Plan(max(sizes), EXPERTS, TOP_K) as plan:
        batches = [Batch(n, 5 + i, plan, *weights) for i, n in enumerate(sizes)]
        want, graphs = [], []
        for b in batches:
            b.step()
            torch.cuda.synchronize()
            want.append(b.results())
        for b in batches[:2]:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                b.step()
        for turn in ((0, 1, 1, 0), (1, 0, 1), (0, 0, 1)):
            for i in turn:
                batches[i].clear()
                graphs[i].replay()
            batches[2].step()
            torch.cuda.synchronize()
            for b, w in zip(batches, want):
                same(b.results(), w, f"{b.rows} rows, turn {turn}")
