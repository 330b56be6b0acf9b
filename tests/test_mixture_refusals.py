"""The block norm's, the router's and the experts' calls refuse bad arguments on the host, before any GPU call
(runs without one: pointers are made-up addresses that are never read)."""
import pytest

from rank_adapter_gemm_lora_amd import binding as lb
from test_mx_refusals import BF, P, _args, refused

NN = ("out", "ldo", "q", "ldq", "s", "lds", "h", "ldh", "y", "ldy", "r", "ldr", "post", "gate", "ldg", "scale", "pre", "eps",
      "dtype", "n", "k")
NB = (P, 104, P, 128, P, 16, P, 104, P, 104, P, 104, P, P, 104, 1.0, P, 1e-5, BF, 4, 104)


@pytest.mark.parametrize("change,status", [
    ({"out": 0, "q": 0, "s": 0, "h": 0}, lb.LORA_E_ARG), ({"q": 0}, lb.LORA_E_ARG), ({"s": 0}, lb.LORA_E_ARG),
    ({"y": 0}, lb.LORA_E_ARG), ({"pre": 0}, lb.LORA_E_ARG), ({"pre": 0, "out": 0}, lb.LORA_E_ARG),
    ({"pre": 0, "q": 0, "s": 0}, lb.LORA_E_ARG), ({"pre": P + 4}, lb.LORA_E_ARG), ({"post": P + 8}, lb.LORA_E_ARG),
    ({"gate": P + 2}, lb.LORA_E_ARG), ({"gate": P + 2, "ldg": 0}, lb.LORA_E_ARG), ({"ldg": 96}, lb.LORA_E_ARG),
    ({"ldg": -104}, lb.LORA_E_ARG), ({"ldg": 108}, lb.LORA_E_ARG), ({"eps": -1.0}, lb.LORA_E_ARG),
    ({"eps": float("nan")}, lb.LORA_E_ARG), ({"scale": float("inf")}, lb.LORA_E_ARG), ({"scale": float("nan")}, lb.LORA_E_ARG),
    ({"ldy": 96}, lb.LORA_E_ARG), ({"ldr": 100}, lb.LORA_E_ARG), ({"ldh": 108}, lb.LORA_E_ARG), ({"ldo": 0}, lb.LORA_E_ARG),
    ({"out": P + 8}, lb.LORA_E_ARG), ({"h": P + 8}, lb.LORA_E_ARG), ({"r": P + 8}, lb.LORA_E_ARG), ({"ldq": 64}, lb.LORA_E_ARG),
    ({"lds": 8}, lb.LORA_E_ARG), ({"k": 12}, lb.LORA_E_ARG), ({"k": 0}, lb.LORA_E_ARG), ({"n": -2}, lb.LORA_E_ARG),
    ({"dtype": 2}, lb.LORA_E_ARG), ({"ldy": 1 << 60}, lb.LORA_E_ARG), ({"n": 1 << 30}, lb.LORA_E_UNSUPPORTED),
    ({"k": (1 << 15) + 8}, lb.LORA_E_UNSUPPORTED),
])
def test_block_norm_refuses(change, status):
    refused(lb.lora_block_norm_mx, _args(NN, NB, change), status)


def test_block_norm_without_rows():
    lb.lora_block_norm_mx(P, 104, 0, 0, 0, 0, 0, 0, 0, 104, 0, 0, 0, 0, 0, 1.0, P, 0.0, BF, 0, 104)


def test_plan_refuses_before_the_device():
    import ctypes
    lib = lb.load()
    out = ctypes.c_void_p()
    assert lib.lora_moe_plan_destroy(None) == lb.LORA_OK
    assert lib.lora_moe_plan_create(None, 8, 4, 2) == lb.LORA_E_ARG
    for rows, experts, top_k in ((0, 4, 2), (-1, 4, 2), (8, 0, 1), (8, 4, 0), (8, 4, 5)):
        assert lib.lora_moe_plan_create(ctypes.byref(out), rows, experts, top_k) == lb.LORA_E_ARG
    for rows, experts, top_k in ((8, 1025, 2), (8, 64, 17), ((1 << 29) + 1, 4, 2)):
        assert lib.lora_moe_plan_create(ctypes.byref(out), rows, experts, top_k) == lb.LORA_E_UNSUPPORTED
    assert lib.lora_moe_route(None, P, P, None, None, P, 8, BF, 4, 0, 1, 1.0, None) == lb.LORA_E_ARG
    assert lib.lora_moe_group(None, P, 4, None, None, None) == lb.LORA_E_ARG
    assert lib.lora_moe_combine(None, P, 64, P, 64, BF, P, None, 0, BF, 64, None) == lb.LORA_E_ARG


def test_fused_product_refuses_without_a_weight():
    assert lb.load().lora_mx_linear_fused(None, P, 64, None, 0, None, 0, BF, P, 128, P, 16, 0, None, 0, None, 0, 1, None) == lb.LORA_E_ARG


def test_experts_refuse_before_the_device():
    import ctypes
    lib = lb.load()
    out = ctypes.c_void_p()
    assert lib.lora_mx_experts_destroy(None) == lb.LORA_OK
    assert lib.lora_mx_experts_create(None, 4, 64, 64, 0) == lb.LORA_E_ARG
    for n, d, k, gated in ((0, 64, 64, 0), (4, 12, 64, 0), (4, 0, 64, 0), (4, 64, 60, 0), (4, 64, 0, 0), (4, 72, 64, 1), (4, 8, 64, 1)):
        assert lib.lora_mx_experts_create(ctypes.byref(out), n, d, k, gated) == lb.LORA_E_ARG
    for n, d, k in ((1025, 64, 64), (4, (1 << 22) + 8, 64), (4, 64, (1 << 20) + 8)):
        assert lib.lora_mx_experts_create(ctypes.byref(out), n, d, k, 0) == lb.LORA_E_UNSUPPORTED
    assert lib.lora_mx_experts_load(None, 0, P, 64, BF, None) == lb.LORA_E_ARG
    assert lib.lora_mx_experts_load_packed(None, 0, P, 64, P, 16, None) == lb.LORA_E_ARG
    assert lib.lora_mx_expert_linear(None, None, P, 64, None, 0, None, 0, BF, P, 128, P, 16, 0, 0, None, 0, None) == lb.LORA_E_ARG
