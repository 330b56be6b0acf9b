"""Every kernel that the products with an epilogue pick: the experts' (groups of uneven sizes, some empty, rows without
an expert) and the fused one.

On 256 CUs the shapes below reach, in turn, for either format: experts 16x64 (8, 4 and 2 wavefronts along k), 32x64 (4 and
2), 64x64 (k in four), 64x128 (k in two; whole), 128x256 or in 4 bits 128x128; fused 16x32, 16x64, 32x64, 64x64, 64x128 (k
split; whole), 128x128 in 4 bits, and the largest tile.

Sums of whole numbers are exact in any order, so ungated outputs are determined.  Gated ones: with exact sums g and u, 16 u
of the value (u = 2^-24) as in test_gpu_mx_experts.py.  Codes are those of the fp32 output, bit for bit: lora_mx_quantize's.
"""
import numpy as np
import pytest
import torch

import mixture_reference as M
import mx_reference as R
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb
from test_gpu_moe import Plan
from test_gpu_mx import DEV, F32, blocks, held, make_weight, stream
from test_gpu_mx_experts import Experts

pytestmark = pytest.mark.gpu

XV = np.array([-2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5, 3.0])
WV = np.array([-6.0, -3.0, -1.0, 0.0, 0.5, 1.0, 2.0, 4.0])


def code_of(v, fmt):
    return R.codes_under(v[None], np.full((1, 1), 127, np.uint8), fmt)[0]


def random_blocks(g, rows, k, values, fmt):
    """(packed codes, padded scales, values) of rows of small whole multiples of 2^-2."""
    i = g.integers(0, len(values), (rows, k))
    s = g.integers(126, 129, (rows, -(-k // 32))).astype(np.uint8)
    v = values[i] * np.repeat(np.exp2(s.astype(float) - 127), 32, axis=1)[:, :k]
    return R.pack(code_of(values, fmt)[i], fmt), R.pad_scales(s, k), torch.from_numpy(v).to(DEV)


def quantised(y, rows, f):
    q, s = blocks(rows, f, R.E4M3, 0, 2)
    lb.lora_mx_quantize(*held(q, s), R.E4M3, y.data_ptr(), y.stride(0), F32, rows, f, stream())
    return q, s


# rows, experts, top_k, k, outputs of the weight
EXPERTS = [(1, 16, 8, 4096, 264), (6, 3, 1, 2056, 520), (9, 3, 2, 136, 1000), (300, 30, 2, 2056, 520), (300, 30, 2, 264, 520),
           (128, 4, 2, 264, 1928), (256, 4, 2, 264, 1928), (512, 4, 2, 264, 1928), (2100, 2, 1, 136, 29184)]


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("gated", (False, True))
@pytest.mark.parametrize("rows,experts,top_k,k,d", EXPERTS)
def test_experts_kernels(rows, experts, top_k, k, d, gated, fmt):
    note(f"experts' kernels {rows} rows top {top_k} of {experts} {k}x{d} gated {gated} format {fmt}")
    g = np.random.default_rng(rows + k + d)
    d = d // 16 * 16 if gated else d
    f = d // 2 if gated else d
    packed, wv = [], []
    for _ in range(experts):
        q, s, v = random_blocks(g, d, k, WV, R.E2M1)
        packed.append((q, s))
        wv.append(v)
    p = np.exp(g.standard_normal(experts))
    p[0] = 0                                           # an expert without rows
    ids = g.choice(experts, (rows, top_k), p=p / p.sum()).astype(np.int32)
    ids[g.random((rows, top_k)) < 0.03] = -1
    order, offsets, _ = M.group(ids, experts)
    n, pairs = int(offsets[-1]), rows * top_k
    xq, xs, xv = random_blocks(g, rows, k, XV, fmt)
    dq, ds, di = torch.from_numpy(xq).to(DEV), torch.from_numpy(xs).to(DEV), torch.from_numpy(ids).to(DEV)
    row = torch.from_numpy(order // top_k).to(DEV).long()
    y = torch.full((pairs + 2, f), 7.0, device=DEV)
    yq, ys = blocks(pairs, f, R.E4M3, 0, 2)
    with Experts(packed, d, k, gated) as x, Plan(rows, experts, top_k) as plan:
        lb.lora_moe_group(plan.at, di.data_ptr(), rows, 0, 0, stream())
        lb.lora_mx_expert_linear(x.at, plan.at, y.data_ptr(), f, *held(yq, ys), F32, *held(dq, ds), fmt, lb.LORA_MOE_ROWS, 0,
                                 lb.LORA_ACT_SWIGLU if gated else lb.LORA_ACT_NONE, stream())
        y2 = torch.full_like(y, 7.0)   # without blocks, the other way of storing
        lb.lora_mx_expert_linear(x.at, plan.at, y2.data_ptr(), f, 0, 0, 0, 0, F32, *held(dq, ds), fmt, lb.LORA_MOE_ROWS, 0,
                                 lb.LORA_ACT_SWIGLU if gated else lb.LORA_ACT_NONE, stream())
        torch.cuda.synchronize()
    assert torch.equal(y, y2)
    assert (y[n:] == 7).all()
    for e in range(experts):
        at = slice(offsets[e], offsets[e + 1])
        v = xv[row[at]] @ wv[e].T
        assert v.numel() == 0 or v.abs().max() < 2 ** 19   # multiples of 2^-4: exact in fp32
        if not gated:
            assert torch.equal(y[at].double(), v), f"expert {e}"
            continue
        gate, up = v[:, :f], v[:, f:]
        want = gate / (1 + torch.exp(-gate)) * up
        assert ((y[at].double() - want).abs() <= 17 * 2.0 ** -24 * want.abs() + 2.0 ** -100).all(), f"expert {e}"
    q, s = quantised(y, n, f)
    assert torch.equal(yq[:n], q[:n]) and torch.equal(ys[:n], s[:n])
    assert torch.equal(yq[n:], blocks(pairs, f, R.E4M3, 0, 2)[0][n:])


FUSED = [(1, 4096, 264), (17, 264, 2056), (40, 264, 4104), (70, 264, 4104), (120, 264, 4104), (250, 136, 4104), (500, 136, 8200),
         (2048, 136, 4096), (4001, 136, 4088)]


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("rows,k,d", FUSED)
def test_fused_kernels(rows, k, d, fmt):
    note(f"fused kernels {rows}x{k}x{d} format {fmt}")
    g = np.random.default_rng(rows + k + d)
    wq, ws, wv = random_blocks(g, d, k, WV, R.E2M1)
    xq, xs, xv = random_blocks(g, rows, k, XV, fmt)
    dq, ds = torch.from_numpy(xq).to(DEV), torch.from_numpy(xs).to(DEV)
    bias = torch.from_numpy(g.integers(-64, 65, d).astype(np.float32)).to(DEV)
    r = torch.from_numpy(g.integers(-256, 257, (rows, d)).astype(np.float32) * 0.5).to(DEV)
    y, y2 = torch.full((rows + 2, d), 7.0, device=DEV), torch.full((rows + 2, d), 7.0, device=DEV)
    yq, ys = blocks(rows, d, R.E4M3, 0, 2)
    w = make_weight(d, k, wq, ws)
    try:
        lb.lora_mx_linear_fused(w, y.data_ptr(), d, *held(yq, ys), F32, *held(dq, ds), fmt, bias.data_ptr(), lb.LORA_ACT_RELU,
                                r.data_ptr(), d, rows, stream())
        lb.lora_mx_linear_fused(w, y2.data_ptr(), d, 0, 0, 0, 0, F32, *held(dq, ds), fmt, 0, lb.LORA_ACT_NONE, 0, 0, rows, stream())
    finally:
        torch.cuda.synchronize()
        lb.lora_mx_weight_destroy(w)
    v = xv @ wv.T
    assert v.abs().max() < 2 ** 18
    assert torch.equal(y2[:rows].double(), v) and (y2[rows:] == 7).all()
    assert torch.equal(y[:rows].double(), (v + bias.double()).clamp(min=0) + r.double()) and (y[rows:] == 7).all()
    q, s = quantised(y, rows, d)
    assert torch.equal(yq, q) and torch.equal(ys, s)
