"""The example layer (4-bit base weights, adapters, norm, SwiGLU) against 64-bit forms, and captured.

Every step is checked from the buffers that it read.  Tolerances, from the roundings
counted before the first run (u = 2^-24; half a bf16 step 2^-8 of the value):
  * a projection: the product's sums (chunks + 32) 2^-23 sum |x w|; y rounded to bf16, the
    delta's sums (k + rank roundings, 2 (k + rank) u of its magnitudes) added, rounded again;
  * norm and SwiGLU: as in their own tests, 2^-18 and 16 u of the value, one rounding each;
  * blocks: the codes lie between those of the exact values moved by that much.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

import mx_reference as R
from gpu_helpers import note

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mx_layer.py")
_spec = importlib.util.spec_from_file_location("mx_layer", _path)
ex = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(ex)

HALF, U = 2.0 ** -8, 2.0 ** -24
K, SLICES, F, RANK, SLOTS, ROWS = 264, [256, 64, 64], 520, 16, 3, 21


def host(t):
    return t.double().cpu().numpy()


def held(b, k):
    return R.values(b.q.cpu().numpy(), b.s.cpu().numpy(), R.E4M3, k)


def check_projection(name, got, x, blocks, weight, adapters, ids, slices):
    k = weight.shape[1]
    wq, ws = R.quantize(host(weight), R.E2M1)
    wv, xv = R.values(wq, ws, R.E2M1, k), held(blocks, k)
    base, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    tol = ((k + 127) // 128 + 32) * 2.0 ** -23 * mag
    delta, dmag = np.zeros_like(base), np.zeros_like(base)
    off = np.cumsum([0] + slices)
    for i, s in enumerate(ids if adapters else []):
        if s < 0:
            continue
        A, B, scale = (host(adapters[name, s][0]), host(adapters[name, s][1]), adapters[name, s][2])
        for q in range(len(slices)):
            c = slice(off[q], off[q + 1])
            delta[i, c] = scale * (B[c] @ (A[q] @ x[i]))
            dmag[i, c] = scale * (np.abs(B[c]) @ (np.abs(A[q]) @ np.abs(x[i])))
    want = base + delta
    tol = tol + HALF * (np.abs(base) + tol) + 2 * (k + RANK) * U * dmag   # y as it is added to
    tol = tol + HALF * (np.abs(want) + tol)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size}"


def check_value(name, got, want, delta):
    bad = ~(np.abs(got - want) <= (HALF * (1 + delta) + delta) * np.abs(want) + 2.0 ** -133)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size}"


def check_blocks(name, blocks, exact, delta, k):
    gs = blocks.s.cpu().numpy()
    n = -(-k // 32)
    lo_s, hi_s = (R.block_scales(exact * f, R.E4M3) for f in (1 - delta, 1 + delta))
    assert ((gs[:, :n] >= lo_s) & (gs[:, :n] <= hi_s)).all(), f"{name}: scales"
    ends = [R.values(R.pack(R.codes_under(exact * f, gs[:, :n], R.E4M3), R.E4M3), gs[:, :n], R.E4M3, k)
            for f in (1 - delta, 1 + delta)]
    got = held(blocks, k)
    assert ((got >= np.minimum(*ends)) & (got <= np.maximum(*ends))).all(), f"{name}: codes"


@pytest.fixture(scope="module")
def case():
    layer, w, adapters = ex.random_layer(K, SLICES, F, ROWS, SLOTS, RANK)
    g = torch.Generator(device="cuda:0").manual_seed(3)
    hidden = torch.randn(ROWS, K, generator=g, device="cuda:0").bfloat16()
    residual = (3 * torch.randn(ROWS, K, generator=g, device="cuda:0")).bfloat16()
    ids = torch.randint(-1, SLOTS, (ROWS,), generator=g, device="cuda:0", dtype=torch.int32)
    yield layer, w, adapters, hidden, residual, ids
    torch.cuda.synchronize()
    layer.close()


def test_layer_steps(case):
    layer, w, adapters, hidden0, residual0, ids = case
    note("mx layer, step by step")
    hidden, residual, who = hidden0.clone(), residual0.clone(), ids.cpu().tolist()
    eps = float(np.float32(layer.eps))

    h, n = R.norm(host(hidden), host(residual), host(w["norm1"]), eps)
    layer.begin(hidden, residual, ids, ROWS)
    check_value("residual", host(residual), h, U)
    check_value("norm1", host(layer.x1), n, 2.0 ** -18)
    check_blocks("norm1", layer.b1, n, 2.0 ** -18, K)
    check_projection("qkv", host(layer.y_qkv), host(layer.x1), layer.b1, w["qkv"], adapters, who, SLICES)

    attention, before = layer.y_qkv[:, :SLICES[0]], residual.clone()
    layer.finish(attention, hidden, residual, ids, ROWS)
    assert np.array_equal(held(layer.bo, SLICES[0]),
                          R.values(*R.quantize(host(attention), R.E4M3), R.E4M3, SLICES[0]))
    check_projection("o", host(layer.y_o), None, layer.bo, w["o"], None, who, [K])
    h, n = R.norm(host(layer.y_o), host(before), host(w["norm2"]), eps)
    check_value("residual", host(residual), h, U)
    check_value("norm2", host(layer.x2), n, 2.0 ** -18)
    check_blocks("norm2", layer.b2, n, 2.0 ** -18, K)
    check_projection("gu", host(layer.y_gu), host(layer.x2), layer.b2, w["gu"], adapters, who, [F, F])
    a = R.swiglu(host(layer.y_gu))
    check_value("swiglu", host(layer.a), a, 16 * U)
    check_blocks("swiglu", layer.ba, a, 16 * U, F)
    check_projection("down", host(hidden), host(layer.a), layer.ba, w["down"], adapters, who, [K])


def test_layer_captured(case):
    """The captured layer on new hidden states, between eager work: the eager bits each time."""
    layer, w, adapters, hidden0, residual0, ids = case
    note("mx layer, captured")
    hidden, residual = hidden0.clone(), residual0.clone()
    layer.step(hidden, residual, ids, ROWS)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(hidden, residual, ids, ROWS)
    for i in range(4):
        h, r = (hidden0 * (1 + i)).contiguous(), (residual0 - i).contiguous()
        hidden.copy_(h)
        residual.copy_(r)
        graph.replay()
        torch.cuda.synchronize()
        layer.step(h, r, ids, ROWS)
        torch.cuda.synchronize()
        assert torch.equal(hidden, h) and torch.equal(residual, r), f"replay {i}"
        assert torch.isfinite(h.float()).all()
