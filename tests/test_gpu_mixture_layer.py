"""The mixture layer of the examples: every step against 64-bit forms of the buffers that it read, and captured.

Tolerances as in the operators' own tests: products (chunks + 32) 2^-23 sum |x w| before their bias (one rounding) and the
rounding to bf16 (2^-8 of the value); adapters as in test_gpu_mx_layer.py; block norms 2^-40 ahead of one rounding; gated
activations, combination and routing weights as in test_gpu_mx_experts.py and test_gpu_moe.py.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import mixture_reference as M
import mx_reference as R
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb
from test_gpu_block_norm import FINE, near, reference
from test_gpu_mx import BF, check_blocks
from test_gpu_mx_fused import check_blocks_within
from test_gpu_mx_layer import held, host

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixture_layer.py")
_spec = importlib.util.spec_from_file_location("mixture_layer", _path)
ex = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(ex)

HALF, U = 2.0 ** -8, 2.0 ** -24
K, SLICES, F, EXPERTS, TOP_K, RANK, SLOTS, ROWS = 264, [256, 64, 64], 136, 12, 3, 16, 3, 37


@pytest.fixture(scope="module")
def case():
    layer, w, adapters = ex.random_layer(K, SLICES, F, EXPERTS, TOP_K, ROWS, SLOTS, RANK)
    g = torch.Generator(device="cuda:0").manual_seed(3)
    x = torch.randn(ROWS, K, generator=g, device="cuda:0").bfloat16()
    residual = (3 * torch.randn(ROWS, K, generator=g, device="cuda:0")).bfloat16()
    ids = torch.randint(-1, SLOTS, (ROWS,), generator=g, device="cuda:0", dtype=torch.int32)
    yield layer, w, adapters, x, residual, ids
    torch.cuda.synchronize()
    layer.close()


def quantised(x):
    blocks = ex.Blocks(ROWS, K, x.device)
    lb.lora_mx_quantize(*blocks.args, ex.E4M3, x.data_ptr(), K, BF, ROWS, K, ex._stream())
    return blocks


def check_norm(y, before, residual, x, blocks, post, pre, eps):
    h, n, size = reference(host(y), host(before), host(post), None, 1.0, host(pre), eps)
    near(host(residual), h, BF, FINE * size, "residual")
    near(host(x), n, BF, FINE * size * np.abs(n / h), "norm")
    check_blocks(blocks.q.cpu().numpy(), blocks.s.cpu().numpy(), n, FINE, K)


def check_qkv(got, x, blocks, w, adapters, who):
    """The sums with their bias rounded to bf16, the adapters' delta added, rounded again: half a step of each."""
    wv, xv = weights_held([w["qkv"]])[0], held(blocks, K)
    base, mag = xv @ wv.T + host(w["bias"]), np.abs(xv) @ np.abs(wv).T
    tol = ((K + 127) // 128 + 32) * 2.0 ** -23 * mag + U * np.abs(base)
    delta, dmag = np.zeros_like(base), np.zeros_like(base)
    off = np.cumsum([0] + SLICES)
    for i, s in enumerate(who):
        if s < 0:
            continue
        A, B, scale = host(adapters["qkv", s][0]), host(adapters["qkv", s][1]), adapters["qkv", s][2]
        for q in range(len(SLICES)):
            c = slice(off[q], off[q + 1])
            delta[i, c] = scale * (B[c] @ (A[q] @ x[i]))
            dmag[i, c] = scale * (np.abs(B[c]) @ (np.abs(A[q]) @ np.abs(x[i])))
    want = base + delta
    tol = tol + HALF * (np.abs(base) + tol) + 2 * (K + RANK) * U * dmag
    tol = tol + HALF * (np.abs(want) + tol)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"qkv: {bad.sum()} of {bad.size}"


def weights_held(w):
    return [R.values(*R.quantize(host(v), R.E2M1), R.E2M1, v.shape[1]) for v in w]


def test_mixture_layer_steps(case):
    layer, w, adapters, x0, residual0, ids = case
    note("mixture layer, step by step")
    x, residual, who, eps = x0.clone(), residual0.clone(), ids.cpu().tolist(), float(np.float32(layer.eps))
    blocks = quantised(x)
    layer.begin(x, blocks, ids, ROWS)
    check_qkv(host(layer.y_qkv), host(x), blocks, w, adapters, who)

    attention, before = layer.y_qkv[:, :SLICES[0]], residual.clone()
    layer.finish(attention, x, blocks, residual, ROWS)
    # the buffers of the middle of the layer, each from what it was made of
    sums = held(layer.bo, SLICES[0]) @ weights_held([w["o"]])[0].T
    mag = np.abs(held(layer.bo, SLICES[0])) @ np.abs(weights_held([w["o"]])[0]).T
    tol = ((SLICES[0] + 127) // 128 + 32) * 2.0 ** -23 * mag
    assert (np.abs(host(layer.y_o) - sums) <= HALF * (np.abs(sums) + tol) + tol).all()
    h1, _, _ = reference(host(layer.y_o), host(before), host(w["post_attention"]), None, 1.0, host(w["pre_mlp"]), eps)
    mid = torch.from_numpy(R.bf16(h1)).to(x.device).bfloat16()
    _, n, size = reference(host(layer.y_o), host(before), host(w["post_attention"]), None, 1.0, host(w["pre_mlp"]), eps)
    near(host(layer.x), n, BF, FINE * size * np.abs(n / h1), "norm")
    check_blocks(layer.bx.q.cpu().numpy(), layer.bx.s.cpu().numpy(), n, FINE, K)

    want_ids, want_w, far = M.route(host(layer.logits), TOP_K, lb.LORA_MOE_SOFTMAX, True, 1.0)
    assert np.array_equal(layer.ids.cpu().numpy(), want_ids)
    assert (np.abs(host(layer.weights) - want_w) <= (far[:, None] + 32) * U * want_w).all()
    order, offsets, place = M.group(want_ids, EXPERTS)
    up, down = weights_held(w["up"]), weights_held(w["down"])
    xv, av = held(layer.bx, K), held(layer.ba, F)
    act, lim = np.zeros((ROWS * TOP_K, F)), np.zeros((ROWS * TOP_K, F))
    y, ylim = np.zeros((ROWS * TOP_K, K)), np.zeros((ROWS * TOP_K, K))
    for e in range(EXPERTS):
        at = slice(offsets[e], offsets[e + 1])
        a = xv[order[at] // TOP_K]
        v, tv = a @ up[e].T, ((K + 127) // 128 + 32) * 2.0 ** -23 * (np.abs(a) @ np.abs(up[e]).T)
        gate, u, tg, tu = v[:, :F], v[:, F:], tv[:, :F], tv[:, F:]
        silu = gate / (1 + np.exp(-gate))
        act[at], lim[at] = silu * u, 1.1 * tg * (np.abs(u) + tu) + np.abs(silu) * tu + 16 * U * np.abs(silu * u)
        y[at] = av[at] @ down[e].T
        ylim[at] = ((F + 127) // 128 + 32) * 2.0 ** -23 * (np.abs(av[at]) @ np.abs(down[e]).T) + U * np.abs(y[at])
    check_blocks_within(layer.ba.q.cpu().numpy(), layer.ba.s.cpu().numpy(), act, lim, F)
    assert (np.abs(host(layer.y) - y) <= ylim).all()
    m, size = M.combine(host(layer.y), place, host(layer.weights), None)
    assert (np.abs(host(layer.m) - m) <= HALF * np.abs(m) + 2 * (TOP_K + 1) * U * size + 2.0 ** -133).all()
    check_norm(layer.m, mid, residual, x, blocks, w["post_mlp"], w["next"], eps)


def test_mixture_layer_captured(case):
    """The captured layer on new hidden states, between eager work: the eager bits each time."""
    layer, _, _, x0, residual0, ids = case
    note("mixture layer, captured")
    x, residual = x0.clone(), residual0.clone()
    blocks = quantised(x)
    layer.step(x, blocks, residual, ids, ROWS)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(x, blocks, residual, ids, ROWS)
    for i in range(4):
        a, r = (x0 * (1 + i)).contiguous(), (residual0 - i).contiguous()
        b = quantised(a)
        x.copy_(a)
        residual.copy_(r)
        blocks.q.copy_(b.q)
        blocks.s.copy_(b.s)
        graph.replay()
        torch.cuda.synchronize()
        layer.step(a, b, r, ids, ROWS)
        torch.cuda.synchronize()
        for got, want in ((x, a), (residual, r), (blocks.q, b.q), (blocks.s, b.s)):
            assert torch.equal(got, want), f"replay {i}"
        assert torch.isfinite(a.float()).all()
