"""The microscaled calls refuse bad arguments on the host, before any GPU call
(runs without one: pointers are made-up addresses that are never read), and the
plain reference's own tables hold."""
import ctypes

import numpy as np
import pytest

import mx_reference as R
from rank_adapter_gemm_lora_amd import binding as lb

P = 0x10000   # a 16-byte aligned address; every call below is refused or has no rows
BF, F32 = lb.LORA_BF16, lb.LORA_F32


def refused(call, args, status):
    with pytest.raises(lb.LoraError) as e:
        call(*args)
    assert e.value.status == status


def _args(names, base, change):
    d = dict(zip(names, base))
    assert set(change) <= set(names)
    d.update(change)
    return [d[n] for n in names]


QN = ("q", "ldq", "s", "lds", "fmt", "x", "ldx", "dtype", "n", "k")
QB = (P, 128, P, 16, R.E4M3, P, 104, BF, 4, 104)
DN = ("x", "ldx", "dtype", "q", "ldq", "s", "lds", "fmt", "n", "k")
DB = (P, 104, BF, P, 128, P, 16, R.E4M3, 4, 104)
BAD = [
    ({"q": 0}, lb.LORA_E_ARG), ({"s": 0}, lb.LORA_E_ARG), ({"x": 0}, lb.LORA_E_ARG),
    ({"q": P + 8}, lb.LORA_E_ARG), ({"s": P + 4}, lb.LORA_E_ARG), ({"x": P + 2}, lb.LORA_E_ARG),
    ({"ldq": 112}, lb.LORA_E_ARG), ({"ldq": 136}, lb.LORA_E_ARG), ({"lds": 8}, lb.LORA_E_ARG),
    ({"lds": 24}, lb.LORA_E_ARG), ({"ldx": 96}, lb.LORA_E_ARG), ({"ldx": 108}, lb.LORA_E_ARG),
    ({"k": 100}, lb.LORA_E_ARG), ({"k": 0}, lb.LORA_E_ARG), ({"k": -8}, lb.LORA_E_ARG),
    ({"n": -1}, lb.LORA_E_ARG), ({"dtype": 2}, lb.LORA_E_ARG), ({"dtype": -1}, lb.LORA_E_ARG),
    ({"fmt": 2}, lb.LORA_E_ARG), ({"ldx": 1 << 60}, lb.LORA_E_ARG), ({"ldq": 1 << 62}, lb.LORA_E_ARG),
    ({"k": (1 << 20) + 8}, lb.LORA_E_UNSUPPORTED), ({"n": 1 << 30}, lb.LORA_E_UNSUPPORTED),
]


@pytest.mark.parametrize("change,status", BAD)
def test_quantize_and_dequantize_refuse(change, status):
    refused(lb.lora_mx_quantize, _args(QN, QB, change), status)
    refused(lb.lora_mx_dequantize, _args(DN, DB, change), status)


NN = ("out", "ldo", "q", "ldq", "s", "lds", "h", "ldh", "x", "ldx", "r", "ldr", "w", "eps", "dtype", "n", "k")
NB = (P, 104, P, 128, P, 16, P, 104, P, 104, P, 104, P, 1e-5, BF, 4, 104)


@pytest.mark.parametrize("change,status", [
    ({"out": 0, "q": 0, "s": 0, "h": 0}, lb.LORA_E_ARG), ({"q": 0}, lb.LORA_E_ARG), ({"s": 0}, lb.LORA_E_ARG),
    ({"x": 0}, lb.LORA_E_ARG), ({"w": 0}, lb.LORA_E_ARG), ({"w": P + 4}, lb.LORA_E_ARG),
    ({"eps": -1.0}, lb.LORA_E_ARG), ({"eps": float("nan")}, lb.LORA_E_ARG), ({"eps": float("inf")}, lb.LORA_E_ARG),
    ({"ldr": 96}, lb.LORA_E_ARG), ({"ldh": 108}, lb.LORA_E_ARG), ({"ldo": 0}, lb.LORA_E_ARG),
    ({"out": P + 8}, lb.LORA_E_ARG), ({"h": P + 8}, lb.LORA_E_ARG), ({"r": P + 8}, lb.LORA_E_ARG),
    ({"ldq": 64}, lb.LORA_E_ARG), ({"k": 12}, lb.LORA_E_ARG), ({"n": -2}, lb.LORA_E_ARG),
    ({"k": (1 << 16) + 8}, lb.LORA_E_UNSUPPORTED),
])
def test_rmsnorm_refuses(change, status):
    refused(lb.lora_rmsnorm_mx, _args(NN, NB, change), status)


SN = ("out", "ldo", "q", "ldq", "s", "lds", "gu", "ldg", "dtype", "n", "f")
SB = (P, 104, P, 128, P, 16, P, 208, BF, 4, 104)


@pytest.mark.parametrize("change,status", [
    ({"out": 0, "q": 0, "s": 0}, lb.LORA_E_ARG), ({"s": 0}, lb.LORA_E_ARG), ({"gu": 0}, lb.LORA_E_ARG),
    ({"ldg": 200}, lb.LORA_E_ARG), ({"ldo": 96}, lb.LORA_E_ARG), ({"f": 20}, lb.LORA_E_ARG),
    ({"dtype": 9}, lb.LORA_E_ARG), ({"f": (1 << 20) + 8}, lb.LORA_E_UNSUPPORTED),
])
def test_swiglu_refuses(change, status):
    refused(lb.lora_swiglu_mx, _args(SN, SB, change), status)


def test_no_rows_do_nothing():
    """Without rows no pointer is needed, and values are still checked."""
    lb.lora_mx_quantize(0, 128, 0, 16, R.E4M3, 0, 104, BF, 0, 104)
    lb.lora_mx_dequantize(0, 104, F32, 0, 64, 0, 16, R.E2M1, 0, 104)
    lb.lora_rmsnorm_mx(P, 104, 0, 0, 0, 0, 0, 0, 0, 104, 0, 0, P, 0.0, BF, 0, 104)
    lb.lora_swiglu_mx(P, 104, 0, 0, 0, 0, 0, 208, F32, 0, 104)
    refused(lb.lora_mx_quantize, (0, 112, 0, 16, R.E4M3, 0, 104, BF, 0, 104), lb.LORA_E_ARG)


def test_weight_refuses_before_the_device():
    lib = lb.load()
    out = ctypes.c_void_p()
    assert lib.lora_mx_weight_destroy(None) == lb.LORA_OK
    assert lib.lora_mx_weight_create(None, 64, 64) == lb.LORA_E_ARG
    for d, k in ((0, 64), (12, 64), (64, 0), (64, 68), (-8, 64)):
        assert lib.lora_mx_weight_create(ctypes.byref(out), d, k) == lb.LORA_E_ARG
    for d, k in (((1 << 22) + 8, 64), (64, (1 << 20) + 8)):
        assert lib.lora_mx_weight_create(ctypes.byref(out), d, k) == lb.LORA_E_UNSUPPORTED
    assert lib.lora_mx_weight_load(None, P, 64, BF, None) == lb.LORA_E_ARG
    assert lib.lora_mx_weight_load_packed(None, P, 64, P, 16, None) == lb.LORA_E_ARG
    assert lib.lora_mx_linear(None, P, 64, BF, P, 128, P, 16, 0, 1, None) == lb.LORA_E_ARG


def test_row_sizes():
    assert [lb.lora_mx_code_bytes(k, R.E4M3) for k in (8, 128, 136, 4096)] == [128, 128, 256, 4096]
    assert [lb.lora_mx_code_bytes(k, R.E2M1) for k in (8, 128, 136, 4096)] == [64, 64, 128, 2048]
    assert [lb.lora_mx_scale_bytes(k) for k in (8, 512, 520, 4096)] == [16, 16, 32, 128]


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
def test_reference_formats(fmt):
    g = R.grid(fmt)
    assert g[-1] == {R.E4M3: 448.0, R.E2M1: 6.0}[fmt] and (np.diff(g) > 0).all()
    if fmt == R.E4M3:
        torch = pytest.importorskip("torch")
        t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
        np.testing.assert_array_equal(g, t)
    # every value of the grid is held exactly; the middle of two goes to the even code
    v = np.zeros((1, 32 * 8))
    n = min(len(g), 31)
    v[0, :n], v[0, 31] = g[-n:], g[-1]
    q, s = R.quantize(v, fmt)
    np.testing.assert_array_equal(R.values(q, s, fmt, v.shape[1])[:, :32], v[:, :32])
    mid = (g[1:] + g[:-1]) / 2
    c = R.codes_under(mid[None], np.full((1, -(-len(mid) // 32)), 127, np.uint8), fmt)[0]
    np.testing.assert_array_equal(c % 2, 0)


def test_reference_special_blocks():
    v = np.zeros((4, 64))
    v[1, 3], v[2, 40], v[3, 0] = np.inf, np.nan, 2.0 ** -140
    q, s = R.quantize(v, R.E4M3)
    assert s[:, :2].tolist() == [[0, 0], [255, 0], [0, 255], [0, 0]] and not q.any()
