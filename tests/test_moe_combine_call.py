"""lora_moe_combine's arguments, with and without the dtype of the pairs' results (no GPU: the library is a stand-in)."""
import pytest

from rank_adapter_gemm_lora_amd import binding as lb

OUT, Y, W, RES, STREAM = 0x7f0000000000, 0x7f0000100000, 0x7f0000200000, 0x7f0000300000, 0x55550000


class Library:
    def lora_moe_combine(self, *args):
        self.args = args
        return lb.LORA_OK


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(lb, "_lib", lib)
    return lib


@pytest.mark.parametrize("stream", (STREAM, 0, None))
@pytest.mark.parametrize("residual,ldr", [(RES, 72), (0, 0)])
@pytest.mark.parametrize("dtype", (lb.LORA_F32, lb.LORA_BF16))
def test_y_dtype_left_out_is_dtype(library, dtype, residual, ldr, stream):
    lb.lora_moe_combine("plan", OUT, 64, Y, 72, W, residual, ldr, dtype, 64, stream)
    assert library.args == ("plan", OUT, 64, Y, 72, dtype, W, residual, ldr, dtype, 64, stream)
    lb.lora_moe_combine("plan", OUT, 64, Y, 72, W, residual, ldr, dtype, 64)
    assert library.args == ("plan", OUT, 64, Y, 72, dtype, W, residual, ldr, dtype, 64, None)


@pytest.mark.parametrize("y_dtype", (lb.LORA_F32, lb.LORA_BF16))
@pytest.mark.parametrize("weights,residual,ldr", [(W, RES, 72), (W, 0, 0), (0, 0, 0)])
def test_y_dtype_given(library, y_dtype, weights, residual, ldr):
    lb.lora_moe_combine("plan", OUT, 64, Y, 72, y_dtype, weights, residual, ldr, lb.LORA_BF16, 64, STREAM)
    assert library.args == ("plan", OUT, 64, Y, 72, y_dtype, weights, residual, ldr, lb.LORA_BF16, 64, STREAM)
    lb.lora_moe_combine("plan", OUT, 64, Y, 72, y_dtype, weights, residual, ldr, lb.LORA_BF16, 64)
    assert library.args == ("plan", OUT, 64, Y, 72, y_dtype, weights, residual, ldr, lb.LORA_BF16, 64, None)
