"""The microscaled operators at the far ends of what include/lora.h promises."""
import numpy as np
import pytest
import torch

import mx_reference as R
import test_gpu_mx as T
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = lb.LORA_BF16, lb.LORA_F32


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("rows,k", [((1 << 26) + 5, 8), ((1 << 24) + 5, 520)])
def test_rmsnorm_more_rows_than_one_launch_takes(rows, k):
    """2^32 threads and more: one wavefront a row, and four.  In place, from x alone; the norm's error before its
    rounding to bf16 is far under 2^-20 of the value."""
    note(f"rmsnorm {rows}x{k} in place")
    g = torch.Generator(device=DEV).manual_seed(k)
    x = torch.randn(rows, k, generator=g, device=DEV, dtype=torch.bfloat16)
    w = torch.ones(k, dtype=torch.bfloat16, device=DEV)
    edge = (((1 << 32) - 1) // (64 if k == 8 else 256)) // 8 * 8   # first row of the second launch
    parts = [slice(0, 999), slice(edge - 500, edge + 2), slice(rows - 3, rows)]
    h = [x[p].double() for p in parts]
    lb.lora_rmsnorm_mx(x.data_ptr(), k, 0, 0, 0, 0, 0, 0, x.data_ptr(), k, 0, 0, w.data_ptr(), 1e-5, BF, rows, k, stream())
    for p, v in zip(parts, h):
        want = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5)
        assert ((x[p].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want.abs()).all()


# Before its rounding, the norm's value is off by what its root loses, 2^-43 (a 24-bit root, one Newton step and the
# step's own remainder), and three times 2^-47 or less (remainders of 2^-23 held in fp32): under 2^-40 in all.
NEAR = 2.0 ** -40


def check_norm(v, w, dt, eps=0.0, r=None):
    """Values, and codes on either side of a border, of rows v (and residual r) against 64 bits."""
    rows, k = v.shape
    x, hx = T.dense(v, dt, 8)
    wt, hw = T.dense(w, dt)
    rt, hr = T.dense(r, dt) if r is not None else (None, None)
    out, h = torch.empty_like(x), torch.empty_like(x)
    q, s = T.blocks(rows, k, R.E4M3)
    lb.lora_rmsnorm_mx(out.data_ptr(), out.stride(0), *T.held(q, s), h.data_ptr(), h.stride(0), x.data_ptr(), x.stride(0),
                       0 if r is None else rt.data_ptr(), k, wt.data_ptr(), eps, dt, rows, k, stream())
    if r is not None:
        hx = (hx + hr).astype(np.float32).astype(np.float64)   # h is fp32
    with np.errstate(invalid="ignore"):   # a row of zeros
        _, want = R.norm(hx, None, hw, float(np.float32(eps)))
    T.check_dense(h[:, :k].double().cpu().numpy(), hx, dt, 0.0, "h")
    T.check_dense(out[:, :k].double().cpu().numpy(), want, dt, NEAR, "out")
    T.check_blocks(q.cpu().numpy(), s.cpu().numpy(), want, NEAR, k)


# from fp32's smallest values over both ends of a fp32 square to its largest
SIZES = [2.0 ** -140, 1e-36, 1e-30, 1e-25, 1e-18, 1e-14, 1e-3, 1e3, 1e14, 1e18, 1e20, 1e25, 1e30, 3e36]


@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("k", (8, 264, 4104))
def test_rmsnorm_rows_of_every_size(k, dt):
    """Without eps a row's size cancels, also where its mean square is outside fp32's range."""
    note(f"rmsnorm rows of every size, k {k} dtype {dt}")
    g = np.random.default_rng(k)
    v = g.choice([-1.0, 1.0], (len(SIZES), k)) * g.uniform(0.25, 4, (len(SIZES), k)) * np.array(SIZES)[:, None]
    w = g.uniform(0.5, 2, (1, k))
    check_norm(v, w, dt)
    check_norm(v, w, dt, r=-0.25 * v)
