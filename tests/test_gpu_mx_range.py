"""The microscaled operators at the far ends of what include/lora.h promises."""
import pytest
import torch

from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = lb.LORA_BF16


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
