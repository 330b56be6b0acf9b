"""lora_mx_expert_linear on the GPU against 64-bit forms.

Tolerances, counted before the first run (u = 2^-24):
  * whole numbers: sums and bias are exact in fp32 in any order, so fp32 outputs and codes are determined.
  * sums of random data: (chunks + 32) 2^-23 sum |x w|, the bias one rounding, activations as in test_gpu_mx_fused.py.
  * g / (1 + exp(-g)) u: the gate's slope is at most 1.1 and its size at most |g|, its own error 16 u; with the bounds tg
    and tu of the sums, 1.1 tg (|u| + tu) + |silu| tu + 16 u |silu u| + 2^-100; the output half a step.
"""
import numpy as np
import pytest
import torch

import mixture_reference as M
import mx_reference as R
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb
from test_gpu_moe import Plan
from test_gpu_mx import BF, DEV, F32, FILL, HALF, TD, blocks, dense, held, rand, stream
from test_gpu_mx_fused import ACTS, U, activate, check_blocks_within

pytestmark = pytest.mark.gpu


class Experts:
    """Weights loaded from packed rows with noise past k."""

    def __init__(self, packed, d, k, gated):
        g = np.random.default_rng(d + k)
        self.at = lb.lora_mx_experts_create(len(packed), d, k, gated)
        for e, (q, s) in enumerate(packed):
            fq = g.integers(0, 256, (d, lb.lora_mx_code_bytes(k, R.E2M1) + 16), dtype=np.uint8)
            fs = g.integers(0, 256, (d, lb.lora_mx_scale_bytes(k) + 16), dtype=np.uint8)
            fq[:, :k // 2], fs[:, :-(-k // 32)] = q[:, :k // 2], s[:, :-(-k // 32)]
            dq, ds = torch.from_numpy(fq).to(DEV), torch.from_numpy(fs).to(DEV)
            lb.lora_mx_experts_load_packed(self.at, e, *held(dq, ds), stream())
            torch.cuda.synchronize()

    def __enter__(self):
        return self

    def __exit__(self, *_):
        torch.cuda.synchronize()
        lb.lora_mx_experts_destroy(self.at)


def choices(g, rows, experts, top_k, kind):
    if kind == "one":          # everything to one expert
        return np.full((rows, top_k), experts // 2, np.int32)
    p = np.exp(1.5 * g.standard_normal(experts))
    ids = g.choice(experts, (rows, top_k), p=p / p.sum()).astype(np.int32)
    ids[g.random((rows, top_k)) < 0.1] = -1
    if kind == "none":
        ids[:] = -1
    return ids


def run(x, plan, q, s, fmt, by_rows, pairs, f, dt, bias=None, act=lb.LORA_ACT_NONE, want_y=True, want_q=True):
    dq, ds = torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)
    y = torch.full((pairs + 2, f + 8), 7.0, dtype=TD[dt], device=DEV)
    yq, ys = blocks(pairs, f, R.E4M3, 16, 2)
    lb.lora_mx_expert_linear(x.at, plan.at, y.data_ptr() if want_y else 0, y.stride(0), *(held(yq, ys) if want_q else (0, 0, 0, 0)), dt,
                             *held(dq, ds), fmt, lb.LORA_MOE_ROWS if by_rows else lb.LORA_MOE_PAIRS,
                             0 if bias is None else bias.data_ptr(), act, stream())
    return y.double().cpu().numpy(), yq.cpu().numpy(), ys.cpu().numpy()


def untouched(y, q, s, n, f, want_y=True, want_q=True):
    cb, sb = lb.lora_mx_code_bytes(f, R.E4M3), lb.lora_mx_scale_bytes(f)
    ny, nq = n if want_y else 0, n if want_q else 0
    assert (y[ny:] == 7).all() and (y[:, f:] == 7).all(), "y outside its rows and columns"
    assert (q[nq:] == FILL).all() and (q[:, cb:] == FILL).all() and (s[nq:] == FILL).all() and (s[:, sb:] == FILL).all()


# tiles of 16 and 32 rows, 64 with k split, 64, 128 (4 bits: 128 too); k and d that end inside tiles
SHAPES = [(1, 4, 2, 136, 40), (1, 16, 8, 4096, 264), (7, 3, 2, 520, 1000), (50, 8, 3, 264, 136), (64, 4, 2, 1032, 264),
          (90, 2, 2, 648, 392), (130, 3, 2, 136, 72), (700, 8, 2, 264, 1352), (2100, 3, 2, 136, 4104)]


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("rows,experts,top_k,k,d", SHAPES)
def test_experts_whole_numbers(rows, experts, top_k, k, d, fmt):
    g = np.random.default_rng(rows + k + d)
    one = np.full((experts, d, -(-k // 32)), 127, np.uint8)
    w = g.choice([-6.0, -3.0, -1.0, 0.0, 0.5, 1.0, 2.0, 4.0], (experts, d, k))
    sw = g.integers(126, 129, one.shape).astype(np.uint8)
    packed = [(R.pack(R.codes_under(w[e], one[e], R.E2M1), R.E2M1), R.pad_scales(sw[e], k)) for e in range(experts)]
    wv = [R.values(q, s, R.E2M1, k) for q, s in packed]
    b, hb = dense(g.integers(-64, 65, (experts, d)).astype(float), F32)
    with Experts(packed, d, k, False) as x, Plan(rows, experts, top_k) as plan:
        for kind, by_rows in (("some", True), ("some", False), ("one", True), ("none", True)):
            note(f"experts exact {rows} rows top {top_k} of {experts} {k}x{d} format {fmt} {kind} by rows {by_rows}")
            ids = choices(g, rows, experts, top_k, kind)
            order, offsets, _ = M.group(ids, experts)
            n, pairs = int(offsets[-1]), rows * top_k
            n_in = rows if by_rows else pairs
            xs = R.pad_scales(g.integers(126, 129, (n_in, -(-k // 32))).astype(np.uint8), k)
            xv = g.choice([-2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5, 3.0], (n_in, k))
            xq = R.pack(R.codes_under(xv, np.full((n_in, -(-k // 32)), 127, np.uint8), fmt), fmt)
            xv = R.values(xq, xs, fmt, k)
            t = torch.from_numpy(ids).to(DEV)
            lb.lora_moe_group(plan.at, t.data_ptr(), rows, 0, 0, stream())
            want = np.zeros((n, d))
            for e in range(experts):
                at = slice(offsets[e], offsets[e + 1])
                want[at] = xv[order[at] // top_k if by_rows else at] @ wv[e].T + hb[e]
            y, q, s = run(x, plan, xq, xs, fmt, by_rows, pairs, d, F32, b)
            untouched(y, q, s, n, d)
            np.testing.assert_array_equal(y[:n, :d], want)
            part = slice(0, min(n, (1 << 17) // d))
            if n:
                want_q, want_s = R.quantize(want[part], R.E4M3)
                np.testing.assert_array_equal(s[part, :want_s.shape[1]], want_s)
                np.testing.assert_array_equal(q[part, :want_q.shape[1]], want_q)
            y, q, s = run(x, plan, xq, xs, fmt, by_rows, pairs, d, BF, want_q=False)
            untouched(y, q, s, n, d, want_q=False)
            for e in range(experts):
                want[offsets[e]:offsets[e + 1]] -= hb[e]
            np.testing.assert_array_equal(y[:n, :d], R.bf16(want))


@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("rows,experts,top_k,k,f", [(1, 8, 4, 4096, 136), (1, 4, 1, 264, 8), (5, 3, 2, 520, 72), (60, 6, 2, 392, 264),
                                                    (50, 2, 2, 1032, 40), (130, 3, 2, 264, 520), (700, 4, 2, 136, 360),
                                                    (2100, 3, 2, 136, 2056)])
def test_gated_experts(rows, experts, top_k, k, f, fmt, dt):
    g = np.random.default_rng(rows + k + f)
    packed = [R.quantize(g.standard_normal((2 * f, k)) * (1.5 * k ** -0.5), R.E2M1) for _ in range(experts)]
    wv = [R.values(q, s, R.E2M1, k) for q, s in packed]
    xq, xs = R.quantize(rand(rows, rows, k, 0.5), fmt)
    xv = R.values(xq, xs, fmt, k)
    b, hb = dense(g.standard_normal((experts, 2 * f)), dt)
    ids = choices(g, rows, experts, top_k, "some")
    ids[0, 0] = 0
    order, offsets, _ = M.group(ids, experts)
    n, pairs = int(offsets[-1]), rows * top_k
    with Experts(packed, 2 * f, k, True) as x, Plan(rows, experts, top_k) as plan:
        t = torch.from_numpy(ids).to(DEV)
        lb.lora_moe_group(plan.at, t.data_ptr(), rows, 0, 0, stream())
        for bias in (True, False):
            note(f"gated experts {rows} rows top {top_k} of {experts} {k}x{f} format {fmt} dtype {dt} bias {bias}")
            want, tol = np.zeros((n, f)), np.zeros((n, f))
            for e in range(experts):
                at = slice(offsets[e], offsets[e + 1])
                a = xv[order[at] // top_k]
                v = a @ wv[e].T + (hb[e] if bias else 0)
                tv = ((k + 127) // 128 + 32) * 2.0 ** -23 * (np.abs(a) @ np.abs(wv[e]).T) + U * np.abs(v)
                gate, up, tg, tu = v[:, :f], v[:, f:], tv[:, :f], tv[:, f:]
                silu = gate / (1 + np.exp(-gate))
                want[at] = silu * up
                tol[at] = 1.1 * tg * (np.abs(up) + tu) + np.abs(silu) * tu + 16 * U * np.abs(silu * up) + 2.0 ** -100
            y, q, s = run(x, plan, xq, xs, fmt, True, pairs, f, dt, b if bias else None, lb.LORA_ACT_SWIGLU)
            untouched(y, q, s, n, f)
            got = y[:n, :f]
            bad = ~(np.abs(got - want) <= HALF[dt] * (np.abs(want) + tol) + tol + 2.0 ** -133)
            assert not bad.any(), f"{bad.sum()} of {bad.size}"
            part = slice(0, min(n, (1 << 17) // f))
            check_blocks_within(q[part], s[part], want[part], tol[part], f)
            y2, q2, s2 = run(x, plan, xq, xs, fmt, True, pairs, f, dt, b if bias else None, lb.LORA_ACT_SWIGLU, want_y=False)
            untouched(y2, q2, s2, n, f, want_y=False)
            assert np.array_equal(q, q2) and np.array_equal(s, s2)


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("rows,experts,top_k,k,d", [(9, 4, 2, 520, 264), (600, 5, 2, 264, 136)])
def test_experts_activations(rows, experts, top_k, k, d, fmt):
    g = np.random.default_rng(rows + k + d)
    packed = [R.quantize(g.standard_normal((d, k)) * (1.5 * k ** -0.5), R.E2M1) for _ in range(experts)]
    wv = [R.values(q, s, R.E2M1, k) for q, s in packed]
    ids = choices(g, rows, experts, top_k, "some")
    order, offsets, _ = M.group(ids, experts)
    n, pairs = int(offsets[-1]), rows * top_k
    xq, xs = R.quantize(rand(rows, pairs, k, 0.5), fmt)
    xv = R.values(xq, xs, fmt, k)
    v, tol = np.zeros((n, d)), np.zeros((n, d))
    for e in range(experts):
        at = slice(offsets[e], offsets[e + 1])
        v[at] = xv[at] @ wv[e].T
        tol[at] = ((k + 127) // 128 + 32) * 2.0 ** -23 * (np.abs(xv[at]) @ np.abs(wv[e]).T)
    with Experts(packed, d, k, False) as x, Plan(rows, experts, top_k) as plan:
        t = torch.from_numpy(ids).to(DEV)
        lb.lora_moe_group(plan.at, t.data_ptr(), rows, 0, 0, stream())
        for act in ACTS:
            note(f"experts {rows} rows top {top_k} of {experts} {k}x{d} format {fmt} act {act}")
            want, own = activate(act, v)
            lim = 1.2 * tol + own
            y, q, s = run(x, plan, xq, xs, fmt, False, pairs, d, F32, None, act)
            untouched(y, q, s, n, d)
            bad = ~(np.abs(y[:n, :d] - want) <= HALF[F32] * np.abs(want) + 2 * lim)
            assert not bad.any(), f"act {act}: {bad.sum()} of {bad.size}"
            check_blocks_within(q, s, want, lim, d)


def test_experts_dense_loads_and_reload():
    """Dense weights as lora_mx_quantize quantises them, gated and not; a reload replaces one expert alone."""
    experts, rows, k, f = 3, 20, 264, 72
    g = np.random.default_rng(0)
    note("experts dense loads")
    for gated in (False, True):
        d = 2 * f if gated else f
        w = [dense(rand(e + 7, d, k, 0.5), BF, 8) for e in range(experts + 1)]
        packed = [R.quantize(h, R.E2M1) for _, h in w]
        xq, xs = R.quantize(rand(3, rows, k, 0.3), R.E4M3)
        ids = torch.from_numpy(np.arange(rows, dtype=np.int32)[:, None] % experts).to(DEV)
        act = lb.LORA_ACT_SWIGLU if gated else lb.LORA_ACT_NONE
        with Experts(packed[:experts], d, k, gated) as x, Plan(rows, experts, 1) as plan:
            lb.lora_moe_group(plan.at, ids.data_ptr(), rows, 0, 0, stream())
            want = run(x, plan, xq, xs, R.E4M3, True, rows, f, F32, None, act)
            y = lb.lora_mx_experts_create(experts, d, k, gated)
            try:
                for e in range(experts):
                    with pytest.raises(lb.LoraError) as err:   # not all are loaded
                        lb.lora_mx_expert_linear(y, plan.at, w[0][0].data_ptr(), 264, 0, 0, 0, 0, BF, w[0][0].data_ptr(), 384,
                                                 w[0][0].data_ptr(), 16, R.E4M3, lb.LORA_MOE_ROWS, 0, act, stream())
                    assert err.value.status == lb.LORA_E_EMPTY
                    lb.lora_mx_experts_load(y, e, w[e][0].data_ptr(), w[e][0].stride(0), BF, stream())
                z = type("Z", (), {"at": y})
                got = run(z, plan, xq, xs, R.E4M3, True, rows, f, F32, None, act)
                assert all(np.array_equal(a, b) for a, b in zip(got, want))
                lb.lora_mx_experts_load(y, 1, w[3][0].data_ptr(), w[3][0].stride(0), BF, stream())
                got = run(z, plan, xq, xs, R.E4M3, True, rows, f, F32, None, act)[0][:rows, :f]
                n = -(-rows // experts)   # group 0; then group 1
                m = -(-(rows - 1) // experts)
                same = (got == want[0][:rows, :f]).all(1)
                assert same[:n].all() and not same[n:n + m].any() and same[n + m:].all()
            finally:
                torch.cuda.synchronize()
                lb.lora_mx_experts_destroy(y)


def test_experts_refusals():
    note("experts refusals")
    t = torch.zeros(256, 256, device=DEV)
    p = t.data_ptr()
    x, gated = lb.lora_mx_experts_create(4, 64, 128, False), lb.lora_mx_experts_create(4, 64, 128, True)
    try:
        with Plan(8, 4, 2) as plan, Plan(8, 5, 2) as other:
            def refused(call, args, status=lb.LORA_E_ARG):
                with pytest.raises(lb.LoraError) as e:
                    call(*args)
                assert e.value.status == status
            for i, v in ((1, -1), (1, 4), (2, 0), (2, p + 8), (3, 120), (3, 132), (4, 2)):
                a = [x, 0, p, 128, F32, stream()]
                refused(lb.lora_mx_experts_load, a[:i] + [v] + a[i + 1:])
            for i, v in ((1, -1), (1, 4), (2, 0), (3, 48), (4, 0), (5, 8)):
                a = [x, 0, p, 64, p, 16, stream()]
                refused(lb.lora_mx_experts_load_packed, a[:i] + [v] + a[i + 1:])
            for e in range(4):
                lb.lora_mx_experts_load(x, e, p, 128, F32, stream())
                lb.lora_mx_experts_load(gated, e, p, 128, F32, stream())
            good = [x, plan.at, p, 64, p, 128, p, 16, F32, p, 128, p, 16, R.E4M3, lb.LORA_MOE_ROWS, p, lb.LORA_ACT_RELU, stream()]
            refused(lb.lora_mx_expert_linear, good, lb.LORA_E_EMPTY)   # nothing grouped yet
            ids = torch.zeros(8, 2, dtype=torch.int32, device=DEV)
            lb.lora_moe_group(plan.at, ids.data_ptr(), 8, 0, 0, stream())
            lb.lora_moe_group(other.at, ids.data_ptr(), 8, 0, 0, stream())
            for i, v in ((0, None), (1, None), (1, other.at), (2, p + 8), (3, 56), (3, 68), (4, 0), (4, p + 8), (5, 64), (6, 0), (7, 8),
                         (8, 2), (9, 0), (10, 112), (11, 0), (12, 8), (13, 2), (14, 2), (15, p + 4), (16, -1),
                         (16, lb.LORA_ACT_SWIGLU), (16, 6)):
                refused(lb.lora_mx_expert_linear, good[:i] + [v] + good[i + 1:])
            refused(lb.lora_mx_expert_linear, good[:2] + [0, 0, 0, 0, 0, 0] + good[8:])
            refused(lb.lora_mx_expert_linear, [gated] + good[1:])      # gated weights have their own activation
            lb.lora_moe_group(plan.at, 0, 0, 0, 0, stream())
            lb.lora_mx_expert_linear(*good[:9], 0, 128, 0, 16, *good[13:])   # no rows: nothing is read
    finally:
        torch.cuda.synchronize()
        lb.lora_mx_experts_destroy(x)
        lb.lora_mx_experts_destroy(gated)


@pytest.mark.parametrize("top_k,experts", [(2, 3), (1, 40)])
def test_experts_under_a_grouping_of_more_rows(top_k, experts):
    """A grouping that was only captured sets the number of rows, not what the plan holds: calls made then stay inside the
    buffers of that number, though the plan's tiles and places go beyond."""
    note(f"experts under a grouping of more rows, top {top_k} of {experts}")
    few, many, k, f = 24, 600, 264, 136
    g = np.random.default_rng(7)
    packed = [R.quantize(g.standard_normal((f, k)), R.E2M1) for _ in range(experts)]
    xq, xs = (torch.from_numpy(t).to(DEV) for t in R.quantize(rand(1, few, k, 0.3), R.E4M3))
    ids = torch.from_numpy(g.integers(0, experts, (many, top_k)).astype(np.int32)).to(DEV)
    y = torch.full((few * top_k + many, f), 7.0, device=DEV)
    out = torch.full((few + many, f), 7.0, device=DEV)
    w = torch.ones(few, top_k, device=DEV)
    with Experts(packed, f, k, False) as x, Plan(many, experts, top_k) as plan:
        def products():
            lb.lora_mx_expert_linear(x.at, plan.at, y.data_ptr(), f, 0, 0, 0, 0, F32, *held(xq, xs), R.E4M3, lb.LORA_MOE_ROWS, 0,
                                     lb.LORA_ACT_NONE, stream())
            lb.lora_moe_combine(plan.at, out.data_ptr(), f, y.data_ptr(), f, F32, w.data_ptr(), 0, 0, F32, f, stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):   # nothing has run yet: no tiles
            lb.lora_moe_group(plan.at, ids.data_ptr(), few, 0, 0, stream())
        lb.lora_mx_expert_linear(x.at, plan.at, y.data_ptr(), f, 0, 0, 0, 0, F32, *held(xq, xs), R.E4M3, lb.LORA_MOE_ROWS, 0,
                                 lb.LORA_ACT_NONE, stream())
        torch.cuda.synchronize()
        assert (y == 7).all()
        lb.lora_moe_group(plan.at, ids.data_ptr(), few, 0, 0, stream())
        products()
        torch.cuda.synchronize()
        want = out[:few].clone()
        lb.lora_moe_group(plan.at, ids.data_ptr(), many, 0, 0, stream())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lb.lora_moe_group(plan.at, ids.data_ptr(), few, 0, 0, stream())
        products()
        torch.cuda.synchronize()
        assert (y[few * top_k:] == 7).all() and (out[few:] == 7).all()
        graph.replay()      # now the plan holds what the calls were made for
        products()
        torch.cuda.synchronize()
        assert torch.equal(out[:few], want)
        assert (y[few * top_k:] == 7).all() and (out[few:] == 7).all()
