"""That the microscaled norm and SwiGLU have the precision that include/lora.h states, on ordinary rows.

Tolerances as derived at test_gpu_mx_range.check_norm: the norm's value before its rounding is within 2^-40 (its sum
is in 64 bits, so the length of a row adds nothing), an output half a step of its type more, a code none but within
2^-40 of a border.  SwiGLU's values are those of fp32 operations one by one: no tolerance.
"""
import numpy as np
import pytest
import torch

import test_gpu_mx as T
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb
from test_gpu_mx_range import check_norm

pytestmark = pytest.mark.gpu

BF, F32 = lb.LORA_BF16, lb.LORA_F32


@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("residual", (True, False))
@pytest.mark.parametrize("rows,k", [(7, 8), (33, 136), (65, 1032), (129, 4096), (17, 8200), (9, 14336), (5, 28672), (3, 65536)])
def test_rmsnorm(rows, k, residual, dt):
    note(f"rmsnorm precision {rows}x{k} dtype {dt} residual {residual}")
    v = T.rand(rows * k, rows, k)
    r = T.rand(rows + k, rows, k) if residual else None
    check_norm(v, 1 + 0.2 * T.rand(5, 1, k, 0.0), dt, 1e-5, r)


@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("seed", (1, 2, 3))
def test_swiglu_is_the_operations_one_by_one(seed, dt):
    """Bit for bit torch's exp, sum, quotient and product in fp32 on the GPU, rounded once."""
    n, f = 256, 4096
    note(f"swiglu bits, seed {seed} dtype {dt}")
    v = T.rand(seed, n, 2 * f, 1.0)
    v[:, :f:7] = np.random.default_rng(seed).uniform(-87, 20, v[:, :f:7].shape)
    x, _ = T.dense(v, dt)
    out = torch.empty(n, f, dtype=T.TD[dt], device=T.DEV)
    lb.lora_swiglu_mx(out.data_ptr(), f, 0, 0, 0, 0, x.data_ptr(), 2 * f, dt, n, f, T.stream())
    g, u = x[:, :f].float(), x[:, f:].float()
    a = g / (1 + torch.exp(-g)) * u
    normal = (a == 0) | ((a.abs() >= 2.0 ** -126) & torch.isfinite(a))
    assert normal.double().mean() > 0.9
    got, want = out.float(), a.to(T.TD[dt]).float()
    assert torch.equal(got[normal], want[normal]), f"{int((got != want)[normal].sum())} of {int(normal.sum())}"
