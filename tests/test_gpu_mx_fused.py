"""lora_mx_linear_fused on the GPU: its sums are lora_mx_linear's bit for bit, its epilogue against 64-bit forms.

Tolerances, from the roundings counted before the first run (u = 2^-24):
  * whole numbers: sums, bias and residual are exact in fp32 in any order, so fp32 outputs and codes are determined.
  * sums of random data: (chunks + 32) 2^-23 sum |x w|, as in test_gpu_mx.py; the bias one rounding.
  * activations: their slopes are at most 1.2; their own error, relative: silu 16 u; gelu, over the whole range, (40 + 2
    v^2) u (an erfc within 32 u at an argument z = v / sqrt 2 known to 2 u, which is worth at most 2 (z^2 + 1) 2 u);
    gelu_tanh exp at an argument known to 8 u of it, (16 + 8 |2 z|) u; results under 2^-100 count as zero.
  * the residual one rounding, and the output half a step.
"""
import numpy as np
import pytest
import torch

import mx_reference as R
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb
from test_gpu_mx import BF, DEV, F32, FILL, HALF, LINEAR, TD, blocks, dense, held, linear, make_weight, rand, stream

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ACTS = (lb.LORA_ACT_NONE, lb.LORA_ACT_RELU, lb.LORA_ACT_SILU, lb.LORA_ACT_GELU, lb.LORA_ACT_GELU_TANH)


def activate(act, v):
    """(value, bound of the fp32 form's own error) in 64 bits."""
    from scipy.special import erfc
    if act == lb.LORA_ACT_RELU:
        return np.where(v < 0, 0.0, v), np.zeros_like(v)
    if act == lb.LORA_ACT_SILU:
        a, e = v / (1 + np.exp(-v)), 16.0
    elif act == lb.LORA_ACT_GELU:
        a, e = 0.5 * v * erfc(-v / np.sqrt(2)), 40 + 2 * v * v
    elif act == lb.LORA_ACT_GELU_TANH:
        z2 = 2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)
        with np.errstate(over="ignore"):
            a, e = v / (1 + np.exp(-z2)), 16 + 8 * np.abs(z2)
    else:
        return v, np.zeros_like(v)
    return a, np.minimum(e * U, 1.0) * np.abs(a) + 2.0 ** -100


def check_blocks_within(got_q, got_s, exact, tol, k):
    """e4m3 blocks written from values within tol of exact."""
    rows, n = exact.shape[0], -(-k // 32)
    gs = got_s[:rows, :n]
    size = np.abs(exact)
    lo_s, hi_s = R.block_scales(np.maximum(size - tol, 0), R.E4M3), R.block_scales(size + tol, R.E4M3)
    assert ((gs >= lo_s) & (gs <= hi_s)).all(), "scale"
    assert not got_s[:rows, n:lb.lora_mx_scale_bytes(k)].any(), "scales past the end"
    lo, hi = (R.values(R.pack(R.codes_under(exact + t, gs, R.E4M3), R.E4M3), gs, R.E4M3, k) for t in (-tol, tol))
    got = R.values(got_q[:rows], gs, R.E4M3, k)
    ok = (got >= lo) & (got <= hi)
    assert ok.all(), f"{(~ok).sum()} codes"
    assert not got_q[:rows, k:lb.lora_mx_code_bytes(k, R.E4M3)].any(), "codes past the end"


def fused(w, q, s, fmt, rows, d, dt, bias=None, act=lb.LORA_ACT_NONE, residual=None, ldr=0, want_y=True, want_q=True, pad=8, guard=2):
    dq, ds = torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)
    y = torch.full((rows + guard, d + pad), 7.0, dtype=TD[dt], device=DEV)
    yq, ys = blocks(rows, d, R.E4M3, 16, guard)
    lb.lora_mx_linear_fused(w, y.data_ptr() if want_y else 0, y.stride(0), *(held(yq, ys) if want_q else (0, 0, 0, 0)), dt,
                            *held(dq, ds), fmt, 0 if bias is None else bias.data_ptr(), act,
                            0 if residual is None else residual.data_ptr(), ldr, rows, stream())
    got, gq, gs = y.double().cpu().numpy(), yq.cpu().numpy(), ys.cpu().numpy()
    cb, sb = lb.lora_mx_code_bytes(d, R.E4M3), lb.lora_mx_scale_bytes(d)
    if not want_y:
        assert (got == 7).all()
    if not want_q:
        assert (gq == FILL).all() and (gs == FILL).all()
    assert (got[rows:] == 7).all() and (got[:, d:] == 7).all(), "y outside its rows and columns"
    assert (gq[rows:] == FILL).all() and (gq[:, cb:] == FILL).all() and (gs[rows:] == FILL).all() and (gs[:, sb:] == FILL).all()
    return got[:rows, :d], gq[:rows, :cb], gs[:rows, :sb]


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("rows,k,d", LINEAR)
def test_fused_whole_numbers(rows, k, d, fmt):
    note(f"fused exact {rows}x{k}x{d} format {fmt}")
    g = np.random.default_rng(rows * 7 + k + d)
    x = g.choice([-2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5, 3.0], (rows, k))
    w = g.choice([-6.0, -3.0, -1.0, 0.0, 0.5, 1.0, 2.0, 4.0], (d, k))
    sx = g.integers(126, 129, (rows, -(-k // 32))).astype(np.uint8)
    sw = g.integers(126, 129, (d, -(-k // 32))).astype(np.uint8)
    one = np.full_like(sx, 127), np.full_like(sw, 127)
    xq, wq = R.pack(R.codes_under(x, one[0], fmt), fmt), R.pack(R.codes_under(w, one[1], R.E2M1), R.E2M1)
    xs, ws = R.pad_scales(sx, k), R.pad_scales(sw, k)
    sums = R.values(xq, xs, fmt, k) @ R.values(wq, ws, R.E2M1, k).T   # multiples of 2^-4 below 2^19: exact
    assert np.abs(sums).max() < 2 ** 19
    b, hb = dense(g.integers(-64, 65, (1, d)).astype(float), BF)
    r, hr = dense(g.integers(-256, 257, (rows, d)) * 0.5, F32, 16)
    h = make_weight(d, k, wq, ws, pad=16)
    try:
        bf = b.float().contiguous()
        for act in (lb.LORA_ACT_NONE, lb.LORA_ACT_RELU):
            want = sums + hb
            want = (np.maximum(want, 0) if act else want) + hr
            y, q, s = fused(h, xq, xs, fmt, rows, d, F32, bf, act, r, r.stride(0))
            np.testing.assert_array_equal(y, want)
            if rows * d <= 1 << 18:
                want_q, want_s = R.quantize(want, R.E4M3)
                np.testing.assert_array_equal(s, want_s)
                np.testing.assert_array_equal(q, want_q)
        y, _, _ = fused(h, xq, xs, fmt, rows, d, BF, b, want_q=False)
        np.testing.assert_array_equal(y, R.bf16(sums + hb))
        # nothing to fuse: the plain product
        y, _, _ = fused(h, xq, xs, fmt, rows, d, BF, want_q=False)
        np.testing.assert_array_equal(y, linear(h, xq, xs, fmt, rows, d, BF))
    finally:
        torch.cuda.synchronize()
        lb.lora_mx_weight_destroy(h)


@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("rows,k,d", [(1, 4096, 520), (3, 264, 40), (21, 512, 1000), (70, 1032, 264), (260, 640, 776), (1100, 136, 392)])
def test_fused_random(rows, k, d, fmt, dt):
    g = np.random.default_rng(rows + k + d)
    xq, xs = R.quantize(rand(rows, rows, k, 0.5), fmt)
    wq, ws = R.quantize(g.standard_normal((d, k)) * (1.5 * k ** -0.5), R.E2M1)
    xv, wv = R.values(xq, xs, fmt, k), R.values(wq, ws, R.E2M1, k)
    sums, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    tol = ((k + 127) // 128 + 32) * 2.0 ** -23 * mag
    b, hb = dense(g.standard_normal((1, d)), dt)
    r, hr = dense(rand(rows + 2, rows, d), dt, 16)
    h = make_weight(d, k, wq, ws)
    try:
        plain = linear(h, xq, xs, fmt, rows, d, F32)
        for act in ACTS:
            note(f"fused random {rows}x{k}x{d} format {fmt} dtype {dt} act {act}")
            v = sums + hb
            a, own = activate(act, v)
            t = 1.2 * (tol + U * np.abs(v)) + own
            want = a + hr
            t = t + U * (np.abs(want) + t)
            y, q, s = fused(h, xq, xs, fmt, rows, d, dt, b, act, r, r.stride(0))
            bad = ~(np.abs(y - want) <= HALF[dt] * (np.abs(want) + t) + t + 2.0 ** -133)
            assert not bad.any(), f"act {act}: {bad.sum()} of {bad.size}"
            check_blocks_within(q, s, want, t, d)
            # without its other outputs, bias and residual: the same bits where they do not enter
            y2, _, _ = fused(h, xq, xs, fmt, rows, d, dt, b, act, r, r.stride(0), want_q=False)
            _, q2, s2 = fused(h, xq, xs, fmt, rows, d, dt, b, act, r, r.stride(0), want_y=False)
            assert np.array_equal(y, y2) and np.array_equal(q, q2) and np.array_equal(s, s2)
        y, _, _ = fused(h, xq, xs, fmt, rows, d, F32, want_q=False)
        np.testing.assert_array_equal(y, plain)
    finally:
        torch.cuda.synchronize()
        lb.lora_mx_weight_destroy(h)


@pytest.mark.parametrize("act", ACTS)
def test_fused_activations_at_the_ends_of_the_range(act):
    """Values given by the bias under a product of zeros: the formula's, infinities and NaN too."""
    note(f"fused ends of the range act {act}")
    v = np.concatenate([[0.0, -0.0, np.inf, -np.inf, np.nan], np.outer([1, -1], [1e-38, 1e-20, 1e-4, 0.5, 3, 8, 12.9, 14, 20, 60, 87, 88.5,
                                                                                 90, 104, 200, 1e4, 1e10, 1e20, 3e38]).ravel()])
    v = np.concatenate([v, np.linspace(-16, 16, 8 * 400)])
    d = -(-len(v) // 8) * 8
    b, hb = dense(np.pad(v, (0, d - len(v)))[None], F32)
    w = make_weight(d, 32, *R.quantize(np.ones((d, 32)), R.E2M1))
    try:
        y, _, _ = fused(w, *R.quantize(np.zeros((1, 32)), R.E4M3), R.E4M3, 1, d, F32, b, act, want_q=False)
    finally:
        torch.cuda.synchronize()
        lb.lora_mx_weight_destroy(w)
    with np.errstate(all="ignore"):
        want, own = activate(act, hb)
    got = y[:, :d]
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    ends = np.isinf(want)
    np.testing.assert_array_equal(got[ends], want[ends])
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= HALF[F32] * np.abs(want) + 2 * own + 2.0 ** -149) & ~np.isnan(want) & ~ends
    assert not bad.any(), hb[bad]


def test_fused_in_place_nan_stream_and_replays():
    rows, k, d = 40, 512, 264
    g = np.random.default_rng(1)
    xq, xs = R.quantize(rand(2, rows, k, 0.5), R.E4M3)
    wq, ws = R.quantize(g.standard_normal((d, k)) * k ** -0.5, R.E2M1)
    xs[3, 2] = 255                       # a row of NaN
    h = make_weight(d, k, wq, ws)
    r, hr = dense(rand(5, rows, d), BF)
    dq, ds = torch.from_numpy(xq).to(DEV), torch.from_numpy(xs).to(DEV)
    yq, ys = blocks(rows, d, R.E4M3)
    try:
        note("fused in place")
        y = r.clone()

        def call():
            lb.lora_mx_linear_fused(h, y.data_ptr(), d, *held(yq, ys), BF, *held(dq, ds), R.E4M3, 0, lb.LORA_ACT_RELU, y.data_ptr(), d,
                                    rows, stream())
        call()
        want, wq2, ws2 = fused(h, xq, xs, R.E4M3, rows, d, BF, None, lb.LORA_ACT_RELU, r, d)
        np.testing.assert_array_equal(y.double().cpu().numpy(), want)
        assert np.isnan(want[3]).all() and np.isfinite(np.delete(want, 3, 0)).all()
        assert (ws2[3, :-(-d // 32)] == 255).all() and not wq2[3].any()
        assert np.array_equal(yq[:rows].cpu().numpy(), wq2) and np.array_equal(ys[:rows].cpu().numpy(), ws2)
        note("fused captured")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            y.copy_(r)
            call()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(y.double().cpu().numpy(), want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for i in range(3):
            y.copy_(r)
            graph.replay()
            torch.cuda.synchronize()
            np.testing.assert_array_equal(y.double().cpu().numpy(), want, err_msg=f"replay {i}")
    finally:
        torch.cuda.synchronize()
        lb.lora_mx_weight_destroy(h)


def test_fused_refusals():
    note("fused refusals")
    t = torch.zeros(256, 256, device=DEV)
    p = t.data_ptr()
    w = lb.lora_mx_weight_create(64, 128)
    try:
        def refused(args, status=lb.LORA_E_ARG):
            with pytest.raises(lb.LoraError) as e:
                lb.lora_mx_linear_fused(*args)
            assert e.value.status == status
        good = [w, p, 64, p, 128, p, 16, F32, p, 128, p, 16, R.E4M3, p, lb.LORA_ACT_GELU, p, 64, 4, stream()]
        refused(good, lb.LORA_E_EMPTY)
        lb.lora_mx_weight_load(w, p, 128, F32, stream())
        for i, v in ((0, 0), (1, p + 8), (2, 56), (2, 68), (3, 0), (3, p + 8), (4, 64), (5, 0), (6, 8), (7, 2), (8, 0), (9, 112), (10, 0),
                     (11, 8), (12, 2), (13, p + 4), (14, -1), (14, lb.LORA_ACT_SWIGLU), (14, 6), (15, p + 8), (16, 56), (17, -1)):
            refused(good[:i] + [v] + good[i + 1:])
        refused(good[:1] + [0, 0, 0, 0, 0, 0] + good[7:])
        refused(good[:17] + [1 << 30] + good[18:], lb.LORA_E_UNSUPPORTED)
        lb.lora_mx_linear_fused(*good[:17], 0, stream())
    finally:
        torch.cuda.synchronize()
        lb.lora_mx_weight_destroy(w)
