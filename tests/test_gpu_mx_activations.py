"""The activations of the products with an epilogue, each to the error that its own operations leave.

Values are given by an fp32 bias under a product of zeros, so that they are any floats and exact.  Errors counted from the
operations before the first run, each at its worst (u = 2^-24; the power of two and the reciprocal are the hardware's,
within one ulp, 2 u; second-order terms are under u / 1000 in all):
  * silu, max(v, 0) - |v| e / (1 + e) with e = exp(-|v|): the power of two 2 u and bringing in what its argument lost u; the
    denominator u, the corrected quotient u, its product with |v| u; of a positive v the tail is at most half and at most
    what is left, so that its 5 u count 5 u at most there; the last sum u: 6 u.  The gate's product one more: 7 u.
  * gelu_tanh, the same with e = exp(-|2 z|): 2 z = v (a + b v^2) with v^2 and b u each, worth less than the whole, the sum of
    products and a u: 3 u of it, which is worth 3 |2 z| u where the logistic falls; 6 u as above.
  * gelu, v Phi(-x) with x = |v| and Phi(-x) = exp(-x^2 / 2) r(x): r's polynomial 1 u; its variable 1 / (1 + 0.3 x) 3 u, worth
    |d log r / d log(1 / (1 + 0.3 x))| times as much, 2.7 at 0 and 1.24 at 13; its sums 4.2 u together, past x = 4 2.7 u;
    times x u, the power of two 2 u and u, the last product and sum u.
Results under 2^-126 are subnormal, or zero where the power of two itself is under 2^-126: 2^-126 there for gelu and
gelu_tanh; silu's are rounded once more, to a multiple of 2^-149.
"""
import numpy as np
import pytest
import torch

import mx_reference as R
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb
from test_gpu_moe import Plan
from test_gpu_mx import DEV, F32, held, make_weight, stream
from test_gpu_mx_experts import Experts

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
K = 32


def values():
    """fp32 values: both signs of every size, and the range where the functions bend, closely."""
    g = np.random.default_rng(5)
    size = np.append(np.exp2(g.uniform(-126, 100, 4095)), 0.0)
    v = np.concatenate([size, -size, np.linspace(-16, 16, 1 << 15), np.linspace(-110, -16, 1 << 13), np.linspace(-13.3, -12.5, 1 << 12),
                        np.linspace(-88.8, -87.2, 1 << 12), np.linspace(-0.02, 0.02, 1 << 11)])
    v = v.astype(np.float32)
    return v[:len(v) // 16 * 16]


def through(act, v):
    """act(v) by the fused product, in fp32."""
    d = len(v)
    w = make_weight(d, K, *R.quantize(np.ones((d, K)), R.E2M1))
    xq, xs = (torch.from_numpy(t).to(DEV) for t in R.quantize(np.zeros((1, K)), R.E4M3))
    b, y = torch.from_numpy(v).to(DEV), torch.empty(1, d, device=DEV)
    try:
        lb.lora_mx_linear_fused(w, y.data_ptr(), d, 0, 0, 0, 0, F32, *held(xq, xs), R.E4M3, b.data_ptr(), act, 0, 0, 1, stream())
    finally:
        torch.cuda.synchronize()
        lb.lora_mx_weight_destroy(w)
    return y[0].double().cpu().numpy()


def within(got, want, relative, absolute):
    assert (np.signbit(got) == np.signbit(want)).all(), "sign, that of a zero too"
    off = np.abs(got - want) - absolute
    worst = np.argmax(off / np.maximum(np.abs(want), 2.0 ** -149) / relative)
    bad = off > relative * U * np.abs(want)
    big = np.abs(want) >= 2.0 ** -126
    print(f"largest error {(np.abs(got - want)[big] / np.abs(want)[big]).max() / U:.2f} u")
    assert not bad.any(), f"{bad.sum()} of {bad.size}, value {got[worst]} for {want[worst]} at {worst}"


def test_silu():
    note("silu to its roundings")
    v = values()
    x = 0.0 + v.astype(np.float64)   # what the sum of zeros and the bias is: -0 becomes 0
    with np.errstate(over="ignore"):
        want = x / (1 + np.exp(-x))
    got = through(lb.LORA_ACT_SILU, v)
    assert (got[(np.abs(want) >= 2.0 ** -126)] != 0).all(), "a value that fp32 holds is flushed"
    within(got, want, 6.01, 2.0 ** -148)


def test_gelu_tanh():
    note("gelu_tanh to its roundings")
    v = values()
    x = 0.0 + v.astype(np.float64)   # what the sum of zeros and the bias is: -0 becomes 0
    z2 = 2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)
    with np.errstate(over="ignore"):
        want = x / (1 + np.exp(-z2))
    fall = 1 / (1 + np.exp(np.minimum(z2, 700)))   # slope of log(1 + exp(-2 z))
    within(through(lb.LORA_ACT_GELU_TANH, v), want, 6.01 + 3 * np.abs(z2) * fall, np.where(np.abs(want) < 2.0 ** -126, 2.0 ** -126, 0.0))


def test_gelu():
    from scipy.special import erfcx, ndtr
    note("gelu to its roundings")
    v = values()
    x = 0.0 + v.astype(np.float64)   # as above
    want = x * ndtr(x)
    size = np.minimum(np.abs(x), 20.0)
    slope = (np.sqrt(2 / np.pi) / erfcx(size / np.sqrt(2)) - size) * (1 + 0.3 * size) / 0.3
    within(through(lb.LORA_ACT_GELU, v), want, 6 + 3 * slope + np.where(size > 4, 2.7, 4.2),
           np.where(np.abs(want) < 2.0 ** -126, 2.0 ** -126, 0.0))


@pytest.mark.parametrize("rows", (1, 64))
def test_gated(rows):
    """silu(g) u of an expert's gate and value; of 64 rows by the kernels that go through LDS."""
    note(f"gated experts to their roundings, {rows} rows")
    g = values()
    f = len(g)
    u = np.random.default_rng(6).standard_normal(f).astype(np.float32)
    zero = R.quantize(np.zeros((2 * f, K)), R.E2M1)
    xq, xs = (torch.from_numpy(t).to(DEV) for t in R.quantize(np.zeros((rows, K)), R.E4M3))
    b, y = torch.from_numpy(np.concatenate([g, u])).to(DEV), torch.empty(rows, f, device=DEV)
    ids = torch.zeros(rows, 1, dtype=torch.int32, device=DEV)
    with Plan(rows, 1, 1) as plan, Experts([zero], 2 * f, K, True) as x:
        lb.lora_moe_group(plan.at, ids.data_ptr(), rows, 0, 0, stream())
        lb.lora_mx_expert_linear(x.at, plan.at, y.data_ptr(), f, 0, 0, 0, 0, F32, *held(xq, xs), R.E4M3, lb.LORA_MOE_ROWS, b.data_ptr(),
                                 lb.LORA_ACT_SWIGLU, stream())
        torch.cuda.synchronize()
    gate, value = 0.0 + g.astype(np.float64), 0.0 + u.astype(np.float64)
    with np.errstate(over="ignore"):
        silu = gate / (1 + np.exp(-gate))
    got = y.double().cpu().numpy()
    assert (got == got[0]).all()
    within(got[0], silu * value, 7.01, 2.0 ** -148 * (1 + np.abs(value)))
