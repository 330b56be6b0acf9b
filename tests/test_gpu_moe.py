"""The router, the grouping by expert and the combination on the GPU against plain forms.

Tolerances, from the roundings counted before the first run (u = 2^-24):
  * ids, order and offsets: none.
  * weights: the difference l - max is rounded once (u of it, which exp turns into u |l - max| of its value); exp within
    4 u; a sum of at most 1024 positive terms, 16 a lane and then 6 steps across lanes, 22 u; sum 1 + exp, quotient,
    normalisation, scale: 4 u.  In all (far + 32) u of the value, far the largest |l| or |l - max| of the row; below
    2^-126 in addition half of the smallest float.
  * combination: one rounding a choice and the residual's: (top_k + 1) u of the magnitudes' sum, then the output's.
"""
import numpy as np
import pytest
import torch

import mixture_reference as M
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb
from test_gpu_mx import BF, DEV, F32, HALF, TD, dense, rand, stream

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SOFTMAX, SIGMOID = lb.LORA_MOE_SOFTMAX, lb.LORA_MOE_SIGMOID


class Plan:
    def __init__(self, rows, experts, top_k):
        self.at = lb.lora_moe_plan_create(max(rows, 1), experts, top_k)
        self.experts, self.top_k = experts, top_k

    def __enter__(self):
        return self

    def __exit__(self, *_):
        torch.cuda.synchronize()
        lb.lora_moe_plan_destroy(self.at)


def logits(seed, rows, experts, dt, special=False, pad=0):
    g = np.random.default_rng(seed)
    x = 2 * g.standard_normal((rows, experts)) + g.standard_normal(experts)
    if special:
        x[g.random((rows, experts)) < 0.1] = -np.inf
        x[g.random((rows, experts)) < 0.05] = np.nan
        put = [np.full(experts, -np.inf), np.zeros(experts), np.where(np.arange(experts) % 2, 0.0, -0.0), np.full(experts, np.nan),
               np.where(np.arange(experts) % 3, 1.0, np.inf), -100.0 - np.arange(experts), 3e38 * np.cos(np.arange(experts)),
               1e-40 * np.sin(np.arange(experts)), np.where(np.arange(experts) == experts - 1, 1.0, -np.inf)]
        for i, row in enumerate(put):
            x[(5 * i) % rows] = row
    t = torch.full((rows, experts + pad), float("inf"), dtype=TD[dt], device=DEV)
    t[:, :experts] = torch.from_numpy(x.astype(np.float32)).to(DEV).to(TD[dt])
    return t, t[:, :experts].double().cpu().numpy()


def route(plan, x, rows, dt, score, renorm, scale=1.0, guard=3):
    n, E, K = x.shape[0] if rows is None else rows, plan.experts, plan.top_k
    ids = torch.full((n + guard, K), 77, dtype=torch.int32, device=DEV)
    w = torch.full((n + guard, K), 7.0, dtype=torch.float32, device=DEV)
    order = torch.full((n * K + guard,), 77, dtype=torch.int32, device=DEV)
    offsets = torch.full((E + 1 + guard,), 77, dtype=torch.int32, device=DEV)
    lb.lora_moe_route(plan.at, ids.data_ptr(), w.data_ptr(), order.data_ptr(), offsets.data_ptr(), x.data_ptr(), x.stride(0), dt, n,
                      score, renorm, scale, stream())
    got = [t.cpu().numpy() for t in (ids, w, order, offsets)]
    assert (got[0][n:] == 77).all() and (got[1][n:] == 7).all() and (got[2][n * K:] == 77).all() and (got[3][E + 1:] == 77).all()
    return got[0][:n], got[1][:n].astype(np.float64), got[2][:n * K], got[3][:E + 1]


def check_route(got, hx, K, score, renorm, scale, what):
    ids, w, order, offsets = got
    want_ids, want_w, far = M.route(hx, K, score, renorm, scale)
    np.testing.assert_array_equal(ids, want_ids, err_msg=what)
    bad = ~(np.abs(w - want_w) <= (far[:, None] + 32) * U * np.abs(want_w) + 2.0 ** -149)
    assert not bad.any(), f"{what}: {bad.sum()} weights"
    want_order, want_offsets, _ = M.group(want_ids, hx.shape[1])
    np.testing.assert_array_equal(order, want_order, err_msg=what)
    np.testing.assert_array_equal(offsets, want_offsets, err_msg=what)


# one and several workgroups, steps that end inside a chunk, every width of the expert groups
SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (16, 16, 16), (64, 64, 8), (129, 60, 4), (200, 128, 8), (300, 65, 7), (257, 256, 8),
          (700, 129, 3), (130, 1000, 16), (90, 1024, 5), (3000, 33, 1), (1500, 257, 11),
          (400, 64, 8), (600, 128, 8), (300, 1024, 8), (5000, 16, 2)]


@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("rows,experts,top_k", SHAPES)
def test_route(rows, experts, top_k, dt):
    with Plan(rows, experts, top_k) as plan:
        for i, (score, renorm, scale) in enumerate([(SOFTMAX, True, 1.0), (SOFTMAX, False, 2.5), (SIGMOID, True, 1.0),
                                                    (SIGMOID, False, -0.5)]):
            special = i % 2 == 0
            what = f"route {rows}x{experts} top {top_k} dtype {dt} score {score} renorm {renorm} special {special}"
            note(what)
            x, hx = logits(rows + experts + i, rows, experts, dt, special, pad=i)
            check_route(route(plan, x, None, dt, score, renorm, scale), hx, top_k, score, renorm, scale, what)


def test_route_of_a_long_batch():
    """More chunks than are counted at once, chunks of several steps, most rows to one expert."""
    rows, experts, top_k = 600_000, 4, 1
    note("route of a long batch")
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn(rows, experts, generator=g, device=DEV)
    x[:, 2] += 3
    with Plan(rows, experts, top_k) as plan:
        ids, w, order, offsets = route(plan, x, None, F32, SOFTMAX, True)
    want = x.argmax(1).cpu().numpy().astype(np.int32)[:, None]   # no two floats of a row are equal here
    assert not (x.sort(1)[0].diff(dim=1) == 0).any()
    np.testing.assert_array_equal(ids, want)
    assert (w == 1).all()
    want_order, want_offsets, _ = M.group(want, experts)
    np.testing.assert_array_equal(order, want_order)
    np.testing.assert_array_equal(offsets, want_offsets)


@pytest.mark.parametrize("rows,experts,top_k", [(5, 3, 2), (400, 24, 4), (4000, 500, 2)])
def test_group_of_given_ids(rows, experts, top_k):
    """Ids out of range are no experts; an expert may be named twice; a plan serves fewer rows than it was made for."""
    g = np.random.default_rng(rows)
    ids = g.integers(-1, experts + 1, (rows, top_k)).astype(np.int32)
    ids[g.random((rows, top_k)) < 0.05] = 2 ** 31 - 1
    ids[g.random((rows, top_k)) < 0.05] = -2 ** 31
    ids[rows // 2] = 1
    note(f"group {rows}x{top_k} of {experts}")
    with Plan(rows + 100, experts, top_k) as plan:
        t = torch.from_numpy(ids).to(DEV)
        for n in (rows, rows // 2, 0, rows):
            order = torch.full((n * top_k + 2,), 77, dtype=torch.int32, device=DEV)
            offsets = torch.full((experts + 3,), 77, dtype=torch.int32, device=DEV)
            lb.lora_moe_group(plan.at, t.data_ptr(), n, order.data_ptr(), offsets.data_ptr(), stream())
            want_order, want_offsets, _ = M.group(ids[:n], experts)
            np.testing.assert_array_equal(order.cpu().numpy(), np.append(want_order, [77, 77]))
            np.testing.assert_array_equal(offsets.cpu().numpy(), np.append(want_offsets, [77, 77]))


@pytest.mark.parametrize("ydt", (BF, F32))
@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("rows,top_k,d", [(1, 1, 8), (3, 2, 520), (70, 8, 1032), (33, 11, 512), (257, 16, 136), (5, 3, 4096)])
def test_combine(rows, top_k, d, dt, ydt):
    experts = 20
    g = np.random.default_rng(rows + d)
    ids = g.integers(-1, experts, (rows, top_k)).astype(np.int32)
    if rows > 2:
        ids[1] = -1    # a row without experts: its residual
    _, _, place = M.group(ids, experts)
    y, hy = dense(rand(rows, rows * top_k, d), ydt, 8)
    y[int((ids >= 0).sum()):] = float("nan")   # rows of pairs without an expert are not read
    hy = y[:, :d].double().cpu().numpy()
    w = torch.from_numpy(g.random((rows, top_k)).astype(np.float32) - 0.3).to(DEV)
    w[torch.from_numpy(ids < 0).to(DEV)] = float("nan")
    r, hr = dense(rand(rows + 1, rows, d), dt, 16)
    note(f"combine {rows}x{d} top {top_k} dtype {dt} of {ydt}")
    with Plan(rows, experts, top_k) as plan:
        t = torch.from_numpy(ids).to(DEV)
        lb.lora_moe_group(plan.at, t.data_ptr(), rows, 0, 0, stream())
        for residual in (None, hr):
            out = torch.full((rows + 1, d + 16), 7.0, dtype=TD[dt], device=DEV)
            lb.lora_moe_combine(plan.at, out.data_ptr(), out.stride(0), y.data_ptr(), y.stride(0), ydt, w.data_ptr(),
                                0 if residual is None else r.data_ptr(), r.stride(0), dt, d, stream())
            got = out.double().cpu().numpy()
            want, size = M.combine(hy, place, w.double().cpu().numpy(), residual)
            bad = ~(np.abs(got[:rows, :d] - want) <= HALF[dt] * np.abs(want) + 2 * (top_k + 1) * U * size + 2.0 ** -133)
            assert not bad.any(), f"{bad.sum()} of {bad.size}"
            assert (got[rows:] == 7).all() and (got[:, d:] == 7).all()
        lb.lora_moe_combine(plan.at, r.data_ptr(), r.stride(0), y.data_ptr(), y.stride(0), ydt, w.data_ptr(), r.data_ptr(),
                            r.stride(0), dt, d, stream())   # in place
        assert torch.equal(r[:, :d], out[:rows, :d])


def test_plan_refusals():
    note("plan refusals")
    t = torch.zeros(64, 64, device=DEV)
    p = t.data_ptr()
    with Plan(8, 6, 2) as plan:
        def refused(call, *args, status=lb.LORA_E_ARG):
            with pytest.raises(lb.LoraError) as e:
                call(*args)
            assert e.value.status == status
        refused(lb.lora_moe_combine, plan.at, p, 64, p, 64, F32, p, 0, 0, F32, 64, stream(), status=lb.LORA_E_EMPTY)
        good = [plan.at, p, p, 0, 0, p, 6, F32, 4, SOFTMAX, True, 1.0, stream()]
        for i, v in ((1, 0), (2, 0), (5, 0), (1, p + 2), (2, p + 1), (3, p + 2), (4, p + 1), (5, p + 2), (6, 5), (6, 1 << 60),
                     (7, 2), (8, -1), (8, 9), (9, 2), (11, float("inf")), (11, float("nan"))):
            refused(lb.lora_moe_route, *good[:i], v, *good[i + 1:])
        refused(lb.lora_moe_group, plan.at, 0, 4, 0, 0, stream())
        refused(lb.lora_moe_group, plan.at, p, 9, 0, 0, stream())
        refused(lb.lora_moe_group, plan.at, p + 2, 4, 0, 0, stream())
        ids = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
        lb.lora_moe_group(plan.at, ids.data_ptr(), 4, 0, 0, stream())
        good = [plan.at, p, 64, p, 64, F32, p, p, 64, F32, 64, stream()]
        for i, v in ((1, 0), (1, p + 4), (2, 56), (2, 60), (3, 0), (4, 56), (5, 2), (6, 0), (6, p + 2), (7, p + 8), (8, 56), (9, 3),
                     (10, 60), (10, 0)):
            refused(lb.lora_moe_combine, *good[:i], v, *good[i + 1:])
        refused(lb.lora_moe_combine, *good[:10], (1 << 22) + 8, stream(), status=lb.LORA_E_UNSUPPORTED)
        torch.cuda.synchronize()


@pytest.mark.parametrize("rows", (40, 2000))
def test_route_replays(rows):
    """A captured router on new logits, with eager work between: the eager results each time."""
    experts, top_k = 64, 8
    note(f"route replays {rows}")
    x, _ = logits(3, rows, experts, BF)
    outs = [torch.empty(rows, top_k, dtype=torch.int32, device=DEV), torch.empty(rows, top_k, device=DEV),
            torch.empty(rows * top_k, dtype=torch.int32, device=DEV), torch.empty(experts + 1, dtype=torch.int32, device=DEV)]
    with Plan(rows, experts, top_k) as plan:
        def call():
            lb.lora_moe_route(plan.at, *(t.data_ptr() for t in outs), x.data_ptr(), experts, BF, rows, SOFTMAX, True, 1.0, stream())
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for i in range(3):
            x.copy_(logits(10 + i, rows, experts, BF)[0])
            graph.replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in outs]
            call()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, outs)), f"replay {i}"
