"""lora_block_norm_mx with weights and gates far from one, whose product leaves fp32's range, and on another stream.

The reference is the formula in 64 bits, which hold every product here; tolerances as in test_gpu_block_norm.py.  An
output past its dtype's largest value is infinite, which the rounding of an exact value there gives too.
"""
import numpy as np
import pytest
import torch

import mx_reference as R
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb
from test_gpu_block_norm import FINE, call, near, reference
from test_gpu_mx import BF, F32, blocks, check_blocks, dense, rand, stream

pytestmark = pytest.mark.gpu


def rounded_past_the_end(v):
    """Values beyond every finite one of bf16 and fp32 as infinities (none of the tests' lies near the border)."""
    assert not ((np.abs(v) > 0.9 * 2.0 ** 128) & (np.abs(v) < 1.1 * 2.0 ** 128)).any()
    return np.where(np.abs(v) >= 2.0 ** 128, np.copysign(np.inf, v), v)


@pytest.mark.parametrize("channel", (True, False))
@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("weight,gate,scale,residual", [
    (70, 70, 1.0, 1.0),          # the product is infinite in fp32, the block's channels of zeros are not
    (66, 62, 2.0 ** -20, 1.0),   # and where the scale brings the value back
    (-80, -75, 2.0 ** 100, 0.0),  # the product is zero in fp32
    (-70, -60, 1.0, 2.0 ** -126),  # and subnormal
    (90, -90, 1.0, 1.0),
])
def test_block_norm_weight_times_gate(weight, gate, scale, residual, dt, channel):
    rows, k = 6, 264
    note(f"block norm weight 2^{weight} gate 2^{gate} scale {scale} dtype {dt} channel {channel}")
    v = rand(3, rows, k, 0.0)
    v[:, ::7] = 0
    y, hy = dense(v, dt)
    r, hr = dense(rand(4, rows, k, 0.0) * residual, dt)
    wp, hp = dense((1 + 0.3 * rand(5, 1, k, 0.0) ** 2) * 2.0 ** weight, dt)
    g, hg = dense((1 + 0.3 * rand(6, 1 if channel else rows, k, 0.0) ** 2) * 2.0 ** gate, dt)
    wn, hn = dense(1 + 0.2 * rand(7, 1, k, 0.0), dt)
    out, h = torch.empty_like(y), torch.empty_like(y)
    q, s = blocks(rows, k, R.E4M3)
    call(rows, k, dt, y, r, wp, g, 0 if channel else k, wn, out, h, q, s, scale=scale, eps=0.0)
    eh, en, size = reference(hy, hr, hp, hg, scale, hn, 0.0)
    near(h.double().cpu().numpy(), rounded_past_the_end(eh), dt, FINE * np.minimum(size, 2.0 ** 128), "h")
    with np.errstate(divide="ignore", invalid="ignore"):
        slack = np.where(eh != 0, FINE * size * np.abs(en / eh), FINE * np.abs(size * hn / np.sqrt((eh * eh).mean(-1, keepdims=True))))
    near(out.double().cpu().numpy(), en, dt, slack, "out")
    check_blocks(q.cpu().numpy(), s.cpu().numpy(), en, FINE, k)


def test_block_norm_on_another_stream():
    """Its bits on a stream of their own are those on the current one."""
    rows, k = 40, 4096
    y, _ = dense(rand(1, rows, k), BF)
    r, _ = dense(rand(2, rows, k), BF)
    w, _ = dense(rand(3, 1, k, 0.0), BF)
    out, h = torch.empty_like(y), torch.empty_like(y)
    q, s = blocks(rows, k, R.E4M3)
    args = (rows, k, BF, y, r, w, w, 0, w, out, h, q, s)
    note("block norm on another stream")
    call(*args)
    torch.cuda.synchronize()
    want = [t.clone() for t in (out, h, q, s)]
    for t in (out, h):
        t.fill_(7.0)
    for t in (q, s):
        t[:rows].fill_(0)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        assert stream() == st.cuda_stream
        call(*args)
    st.synchronize()
    for got, t in zip((out, h, q, s), want):
        assert torch.equal(got, t)
