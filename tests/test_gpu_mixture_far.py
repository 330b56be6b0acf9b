"""Rows far apart: byte offsets past 32 bits in every matrix give the bits of the same rows side by side."""
import numpy as np
import pytest
import torch

import mx_reference as R
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb
from test_gpu_moe import Plan, logits
from test_gpu_mx import BF, DEV, blocks, dense, held, make_weight, rand, stream
from test_gpu_mx_experts import Experts

pytestmark = pytest.mark.gpu

ROWS, FAR = 1100, 1 << 21   # 1100 rows of 2^21 bf16: 4.6 GB


def far(t):
    """t's rows, FAR elements apart."""
    out = torch.empty(t.shape[0], FAR, dtype=t.dtype, device=DEV)[:, :t.shape[1]]
    out.copy_(t)
    return out


def test_block_norm_far():
    note("block norm far")
    k = 264
    y, r, g = (dense(rand(i, ROWS, k), BF)[0] for i in range(3))
    w = dense(rand(3, 1, k, 0.0), BF)[0]

    def run(y, r, g, out, h):
        q, s = blocks(ROWS, k, R.E4M3)
        lb.lora_block_norm_mx(out.data_ptr(), out.stride(0), *held(q, s), h.data_ptr(), h.stride(0), y.data_ptr(), y.stride(0),
                              r.data_ptr(), r.stride(0), w.data_ptr(), g.data_ptr(), g.stride(0), 0.5, w.data_ptr(), 1e-5, BF, ROWS, k,
                              stream())
        return out, h, q, s
    want = run(y, r, g, torch.empty_like(y), torch.empty_like(y))
    got = run(far(y), far(r), far(g), far(y), far(y))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_route_far():
    note("route far")
    experts, top_k = 24, 3
    x, _ = logits(1, ROWS, experts, BF)
    with Plan(ROWS, experts, top_k) as plan:
        def run(x):
            ids = torch.empty(ROWS, top_k, dtype=torch.int32, device=DEV)
            w = torch.empty(ROWS, top_k, device=DEV)
            lb.lora_moe_route(plan.at, ids.data_ptr(), w.data_ptr(), 0, 0, x.data_ptr(), x.stride(0), BF, ROWS, lb.LORA_MOE_SOFTMAX,
                              True, 1.0, stream())
            return ids, w
        want, got = run(x), run(far(x))
        torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows", (30, ROWS))
def test_products_far(rows):
    """X, residual, outputs and the combination's matrices."""
    note(f"products far {rows}")
    k, d, experts = 264, 136, 5
    far_rows = FAR * ROWS // rows // 64 * 64   # as many bytes apart in all
    g = np.random.default_rng(2)
    wq = [R.quantize(g.standard_normal((d, k)), R.E2M1) for _ in range(experts)]
    xq, xs = (torch.from_numpy(t).to(DEV) for t in R.quantize(rand(4, rows, k, 0.3), R.E4M3))
    r = dense(rand(5, rows, d), BF)[0]
    ids = torch.from_numpy(g.integers(-1, experts, (rows, 1)).astype(np.int32)).to(DEV)
    weights = torch.rand(rows, 1, device=DEV)

    def apart(t, n):
        out = torch.empty(t.shape[0], n, dtype=t.dtype, device=DEV)[:, :t.shape[1]]
        out.copy_(t)
        return out
    weight = make_weight(d, k, *wq[0])
    with Experts(wq, d, k, False) as x, Plan(rows, experts, 1) as plan:
        lb.lora_moe_group(plan.at, ids.data_ptr(), rows, 0, 0, stream())

        def run(xq, xs, r, y, yq, ys, z, out):
            lb.lora_mx_linear_fused(weight, y.data_ptr(), y.stride(0), *held(yq, ys), BF, *held(xq, xs), R.E4M3, 0, lb.LORA_ACT_GELU,
                                    r.data_ptr(), r.stride(0), rows, stream())
            lb.lora_mx_expert_linear(x.at, plan.at, z.data_ptr(), z.stride(0), 0, 0, 0, 0, BF, *held(xq, xs), R.E4M3, lb.LORA_MOE_ROWS,
                                     0, lb.LORA_ACT_NONE, stream())
            lb.lora_moe_combine(plan.at, out.data_ptr(), out.stride(0), z.data_ptr(), z.stride(0), BF, weights.data_ptr(), r.data_ptr(),
                                r.stride(0), BF, d, stream())
            return y, yq, ys, z, out
        cb, sb = lb.lora_mx_code_bytes(d, R.E4M3), lb.lora_mx_scale_bytes(d)
        z0 = torch.zeros(rows, d, dtype=torch.bfloat16, device=DEV)
        q0, s0 = (torch.zeros(rows, n, dtype=torch.uint8, device=DEV) for n in (cb, sb))
        want = run(xq, xs, r, z0.clone(), q0.clone(), s0.clone(), z0.clone(), z0.clone())
        got = run(apart(xq, 2 * far_rows), apart(xs, 2 * far_rows), apart(r, far_rows), apart(z0, far_rows), apart(q0, 2 * far_rows),
                  apart(s0, 2 * far_rows), apart(z0, far_rows), apart(z0, far_rows))
        torch.cuda.synchronize()
    lb.lora_mx_weight_destroy(weight)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
