"""The microscaled operators on the GPU against plain 64-bit forms.

Tolerances, from the roundings counted before the first run (u = 2^-24):
  * quantise, dequantise, weight loads: none -- the results are determined.
  * an output in bf16 / fp32 is rounded once: half a step, 2^-8 / 2^-24 of the value.
  * norm in fp32: h = x + r one rounding; the squares and their sum, pairs first and
    then across a thread's at most 64 values, 6 exchange steps and at most 16 wavefronts,
    under 90 roundings, halved by the square root; mean, eps, root, quotient and two
    products: in all under 64 u = 2^-18 of the value.
  * swiglu in fp32: exp within 2 u of its value, sum, quotient, product: under 16 u.
  * blocks of a norm or swiglu: the codes lie between those of the exact values moved down
    and up by that fp32 error (a value next to a border may fall on either side).
  * product: a term is exact; each matrix-core instruction rounds its sum (2^-23 of the
    summed magnitudes allowed, so truncation is covered), one instruction per 128 k, and
    the partial sums of a split are added likewise: (chunks + 32) 2^-23 sum |x w|.
"""
import numpy as np
import pytest
import torch

import mx_reference as R
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = lb.LORA_BF16, lb.LORA_F32
TD = {BF: torch.bfloat16, F32: torch.float32}
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
FILL = 0x5A   # what untouched bytes hold


def stream():
    return torch.cuda.current_stream().cuda_stream


def dense(v, dt, pad=0):
    """Values [rows, k] on the GPU in dtype, in rows of k + pad elements; and the values as held."""
    rows, k = v.shape
    t = torch.full((rows, k + pad), 7.0, dtype=TD[dt], device=DEV)
    t[:, :k] = torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(DEV).to(TD[dt])
    return t, t[:, :k].double().cpu().numpy()


def blocks(rows, k, fmt, pad=0, n_guard=1):
    q = torch.full((rows + n_guard, lb.lora_mx_code_bytes(k, fmt) + pad), FILL, dtype=torch.uint8, device=DEV)
    s = torch.full((rows + n_guard, lb.lora_mx_scale_bytes(k) + pad), FILL, dtype=torch.uint8, device=DEV)
    return q, s


def held(q, s):
    return (q.data_ptr(), q.stride(0), s.data_ptr(), s.stride(0))


def rand(seed, rows, k, spread=2.0):
    g = np.random.default_rng(seed)
    v = g.standard_normal((rows, k)) * np.exp(spread * g.standard_normal((rows, 1)))
    v[:, g.integers(0, k, max(1, k // 64))] *= 30
    v[g.random((rows, k)) < 0.05] = 0
    return v


def specials(v):
    """Put blocks of zeros, infinities, NaN, tiny and huge values into rows of v."""
    rows, k = v.shape
    put = [0.0, np.inf, -np.inf, np.nan, 2.0 ** -133, -(2.0 ** -126), 3e38, 2.0 ** -120]
    for i, p in enumerate(put):
        r, c = i % rows, (37 * i) % k
        if p == 0.0:
            v[r, c // 32 * 32:c // 32 * 32 + 32] = 0
        else:
            v[r, c] = p
            if abs(p) < 1:
                b = c // 32 * 32
                v[r, b:b + 32] = p * np.linspace(-1, 1, 32)[:len(v[r, b:b + 32])]
    return v


SHAPES = [(1, 8), (3, 40), (1, 128), (2, 136), (17, 512), (5, 520), (33, 1032), (65, 4096), (2, 28672)]


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("rows,k", SHAPES)
def test_quantize(rows, k, dt, fmt):
    note(f"quantize {rows}x{k} dtype {dt} format {fmt}")
    for pad, v in ((0, rand(rows + k, rows, k)), (16, specials(rand(rows + 2 * k, rows, k)))):
        x, held_x = dense(v, dt, pad)
        q, s = blocks(rows, k, fmt, pad)
        lb.lora_mx_quantize(*held(q, s), fmt, x.data_ptr(), x.stride(0), dt, rows, k, stream())
        want_q, want_s = R.quantize(held_x, fmt)
        got_q, got_s = q.cpu().numpy(), s.cpu().numpy()
        np.testing.assert_array_equal(got_s[:rows, :want_s.shape[1]], want_s)
        np.testing.assert_array_equal(got_q[:rows, :want_q.shape[1]], want_q)
        for got, want in ((got_q, want_q), (got_s, want_s)):   # nothing else was written
            assert (got[rows:] == FILL).all() and (got[:, want.shape[1]:] == FILL).all()


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("rows,k", [(1, 8), (3, 136), (17, 4104)])
def test_dequantize_all_codes_and_scales(rows, k, dt, fmt):
    note(f"dequantize {rows}x{k} dtype {dt} format {fmt}")
    g = np.random.default_rng(k)
    q = g.integers(0, 256, (rows, lb.lora_mx_code_bytes(k, fmt)), dtype=np.uint8)
    s = g.integers(0, 256, (rows, lb.lora_mx_scale_bytes(k)), dtype=np.uint8)
    s[:, 0] = 255
    dq, ds = torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)
    x = torch.full((rows + 1, k + 8), 7.0, dtype=TD[dt], device=DEV)
    lb.lora_mx_dequantize(x.data_ptr(), x.stride(0), dt, *held(dq, ds), fmt, rows, k, stream())
    want = torch.from_numpy(R.values(q, s, fmt, k)).float().to(TD[dt]).double().numpy()   # rounded once
    got = x.double().cpu().numpy()
    np.testing.assert_array_equal(got[:rows, :k], want)
    assert (got[rows:] == 7).all() and (got[:, k:] == 7).all()


def check_blocks(got_q, got_s, exact, delta, k):
    """Blocks written from fp32 values within delta (relative) of exact."""
    rows = exact.shape[0]
    n = -(-k // 32)
    lo_s, hi_s = (R.block_scales(exact * f, R.E4M3) for f in (1 - delta, 1 + delta))
    gs = got_s[:rows, :n]
    assert ((gs >= lo_s) & (gs <= hi_s)).all(), "scale"
    assert not got_s[:rows, n:lb.lora_mx_scale_bytes(k)].any(), "scales past k"
    ends = [R.values(R.pack(R.codes_under(exact * f, gs, R.E4M3), R.E4M3), gs, R.E4M3, k) for f in (1 - delta, 1 + delta)]
    got = R.values(got_q[:rows], gs, R.E4M3, k)
    lo, hi = np.minimum(*ends), np.maximum(*ends)
    ok = ((got >= lo) & (got <= hi)) | (np.isnan(got) & np.isnan(lo))
    assert ok.all(), f"{(~ok).sum()} codes"
    assert not got_q[:rows, k:lb.lora_mx_code_bytes(k, R.E4M3)].any(), "codes past k"


def check_dense(got, exact, dt, delta, what):
    bad = ~(np.abs(got - exact) <= (HALF[dt] * (1 + delta) + delta) * np.abs(exact) + 2.0 ** -133)
    bad &= ~(np.isnan(got) & np.isnan(exact))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}"


@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("residual", (True, False))
@pytest.mark.parametrize("rows,k", SHAPES + [(3, 2056), (2, 8200), (1, 16392), (2, 65536)])
def test_rmsnorm(rows, k, residual, dt):
    note(f"rmsnorm {rows}x{k} dtype {dt} residual {residual}")
    v = rand(rows + k, rows, k)
    if rows > 2:
        v[1] = 0   # a row of zeros, kept finite by eps
    x, hx = dense(v, dt, 8)
    r, hr = dense(rand(7 * rows + k, rows, k) if rows < 3 else np.where(v == v[1], 0, v * 0.5), dt, 16)
    w, hw = dense(1 + 0.2 * rand(5, 1, k, 0.0), dt)
    out, h = torch.empty_like(x), torch.empty_like(r)
    q, s = blocks(rows, k, R.E4M3, 16)
    lb.lora_rmsnorm_mx(out.data_ptr(), out.stride(0), *held(q, s), h.data_ptr(), h.stride(0), x.data_ptr(), x.stride(0),
                       r.data_ptr() if residual else 0, r.stride(0), w.data_ptr(), 1e-5, dt, rows, k, stream())
    eh, en = R.norm(hx, hr if residual else None, hw, float(np.float32(1e-5)))
    check_dense(h[:, :k].double().cpu().numpy(), eh, dt, 2.0 ** -24, "h")
    check_dense(out[:, :k].double().cpu().numpy(), en, dt, 2.0 ** -18, "out")
    gq, gs = q.cpu().numpy(), s.cpu().numpy()
    check_blocks(gq, gs, en, 2.0 ** -18, k)
    assert (gq[rows:] == FILL).all() and (gq[:, lb.lora_mx_code_bytes(k, R.E4M3):] == FILL).all()
    assert (gs[rows:] == FILL).all() and (gs[:, lb.lora_mx_scale_bytes(k):] == FILL).all()


def test_rmsnorm_in_place_outputs_left_out_and_special_rows():
    rows, k = 5, 264
    v = rand(3, rows, k)
    v[0], v[1, 5], v[2, 9] = 0, np.nan, np.inf
    x, hx = dense(v, BF)
    r, hr = dense(np.zeros((rows, k)), BF)
    w, hw = dense(np.ones((1, k)), BF)
    note("rmsnorm in place")
    # h over the residual and out over x; no blocks
    lb.lora_rmsnorm_mx(x.data_ptr(), k, 0, 0, 0, 0, r.data_ptr(), k, x.data_ptr(), k, r.data_ptr(), k, w.data_ptr(), 0.0,
                       BF, rows, k, stream())
    got = x.double().cpu().numpy()
    with np.errstate(all="ignore"):
        eh, en = R.norm(hx, hr, hw, 0.0)
    assert np.isnan(got[0]).all() and np.isnan(got[1]).all()     # 0 / 0; a NaN takes its row
    assert np.isnan(got[2, 9]) and (got[2, :9] == 0).all()       # inf / inf, the rest over inf
    check_dense(got[3:], en[3:], BF, 2.0 ** -18, "out")
    np.testing.assert_array_equal(r.double().cpu().numpy()[3:], hx[3:])
    # blocks alone, from rows that are not finite
    x, hx = dense(v, BF)
    q, s = blocks(rows, k, R.E4M3)
    lb.lora_rmsnorm_mx(0, 0, *held(q, s), 0, 0, x.data_ptr(), k, 0, 0, w.data_ptr(), 0.0, BF, rows, k, stream())
    gs = s.cpu().numpy()
    assert (gs[:2, :9] == 255).all() and not q.cpu().numpy()[:2].any()
    assert gs[2, 0] == 255 and (gs[2, 1:9] == 0).all()
    check_blocks(q.cpu().numpy()[3:], gs[3:], en[3:], 2.0 ** -18, k)


@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("rows,f", SHAPES)
def test_swiglu(rows, f, dt):
    note(f"swiglu {rows}x{f} dtype {dt}")
    v = rand(rows + f, rows, 2 * f, 0.5)
    v[0, 0], v[-1, -1] = -60.0, 1e4
    x, hx = dense(v, dt, 8)
    out = torch.full((rows + 1, f + 8), 7.0, dtype=TD[dt], device=DEV)
    q, s = blocks(rows, f, R.E4M3)
    lb.lora_swiglu_mx(out.data_ptr(), out.stride(0), *held(q, s), x.data_ptr(), x.stride(0), dt, rows, f, stream())
    with np.errstate(over="ignore"):
        ex = R.swiglu(hx)
    got = out.double().cpu().numpy()
    # exp(-g) past the float range: the quotient is 0 where the exact value is under 2^-126 |g u|
    small = np.abs(ex) < 2.0 ** -100
    check_dense(np.where(small, ex, got[:rows, :f]), ex, dt, 16 * 2.0 ** -24, "out")
    assert (np.abs(got[:rows, :f][small]) < 2.0 ** -99).all()
    assert (got[rows:] == 7).all() and (got[:, f:] == 7).all()
    check_blocks(q.cpu().numpy(), s.cpu().numpy(), ex, 16 * 2.0 ** -24, f)


def make_weight(d, k, q, s, pad=0):
    """A weight loaded from packed rows; what the rows hold past k is noise."""
    g = np.random.default_rng(d + k)
    fq = g.integers(0, 256, (d, lb.lora_mx_code_bytes(k, R.E2M1) + pad), dtype=np.uint8)
    fs = g.integers(0, 256, (d, lb.lora_mx_scale_bytes(k) + pad), dtype=np.uint8)
    fq[:, :k // 2], fs[:, :-(-k // 32)] = q[:, :k // 2], s[:, :-(-k // 32)]
    dq, ds = torch.from_numpy(fq).to(DEV), torch.from_numpy(fs).to(DEV)
    w = lb.lora_mx_weight_create(d, k)
    lb.lora_mx_weight_load_packed(w, *held(dq, ds), stream())
    torch.cuda.synchronize()
    return w


def linear(w, q, s, fmt, rows, d, dt, pad=0, guard=2):
    dq, ds = torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV)
    y = torch.full((rows + guard, d + pad), 7.0, dtype=TD[dt], device=DEV)
    lb.lora_mx_linear(w, y.data_ptr(), y.stride(0), dt, *held(dq, ds), fmt, rows, stream())
    got = y.double().cpu().numpy()
    assert (got[rows:] == 7).all() and (got[:, d:] == 7).all(), "wrote outside its rows and columns"
    return got[:rows, :d]


# rows around every tile height, features and k that end inside tiles, long and short k
LINEAR = [(1, 8, 8), (1, 4096, 256), (2, 136, 24), (15, 520, 72), (16, 2048, 128), (17, 264, 1000), (33, 1032, 40),
          (48, 384, 264), (64, 640, 520), (65, 1152, 248), (100, 4104, 136), (128, 896, 512), (129, 128, 272),
          (192, 1408, 384), (256, 512, 256), (257, 648, 776), (300, 2568, 1032), (511, 4096, 264), (700, 136, 2056),
          (1025, 392, 520), (4100, 264, 136)]


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("rows,k,d", LINEAR)
def test_linear_whole_numbers(rows, k, d, fmt):
    """Codes and scales whose sums are exact in fp32 in any order: every bit has to be right."""
    note(f"linear exact {rows}x{k}x{d} format {fmt}")
    g = np.random.default_rng(rows * 7 + k + d)
    x = g.choice([-2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5, 3.0], (rows, k))
    w = g.choice([-6.0, -3.0, -1.0, 0.0, 0.5, 1.0, 2.0, 4.0], (d, k))
    sx = g.integers(126, 129, (rows, -(-k // 32))).astype(np.uint8)
    sw = g.integers(126, 129, (d, -(-k // 32))).astype(np.uint8)
    one = np.full_like(sx, 127), np.full_like(sw, 127)
    xq = R.pack(R.codes_under(x, one[0], fmt), fmt)
    wq = R.pack(R.codes_under(w, one[1], R.E2M1), R.E2M1)
    xs, ws = R.pad_scales(sx, k), R.pad_scales(sw, k)
    want = R.values(xq, xs, fmt, k) @ R.values(wq, ws, R.E2M1, k).T   # multiples of 2^-4 below 2^20: exact
    assert np.abs(want).max() < 2 ** 19
    h = make_weight(d, k, wq, ws, pad=16)
    try:
        np.testing.assert_array_equal(linear(h, xq, xs, fmt, rows, d, F32, pad=8), want)
        np.testing.assert_array_equal(linear(h, xq, xs, fmt, rows, d, BF, pad=16), R.bf16(want))
    finally:
        lb.lora_mx_weight_destroy(h)


# One size for every tile that the launcher chooses between (256 CUs): rows and features that end inside a tile,
# k that ends inside a chunk, a stage of two chunks and a run of four, more wavefront sets than runs of four.
LINEAR_TILES = [(7, 264, 16000), (24, 1416, 4096), (33, 2312, 4000), (70, 904, 5000), (256, 1416, 4000), (250, 136, 4096),
                (500, 2312, 4040), (1000, 904, 4600), (4000, 392, 2112), (8190, 648, 4088)]


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("rows,k,d", LINEAR_TILES)
def test_linear_whole_numbers_every_tile(rows, k, d, fmt):
    test_linear_whole_numbers(rows, k, d, fmt)


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("rows,k,d", [(1, 4096, 512), (16, 14336, 264), (60, 8192, 264), (250, 4104, 512), (600, 2056, 776)])
def test_linear_hidden_states(rows, k, d, dt, fmt):
    note(f"linear {rows}x{k}x{d} dtype {dt} format {fmt}")
    xq, xs = R.quantize(rand(rows, rows, k), fmt)
    wd, hw = dense(0.02 * rand(d, d, k, 0.3), BF, 8)
    h = lb.lora_mx_weight_create(d, k)
    try:
        lb.lora_mx_weight_load(h, wd.data_ptr(), wd.stride(0), BF, stream())
        got = linear(h, xq, xs, fmt, rows, d, dt)
    finally:
        lb.lora_mx_weight_destroy(h)
    wq, ws = R.quantize(hw, R.E2M1)
    xv, wv = R.values(xq, xs, fmt, k), R.values(wq, ws, R.E2M1, k)
    want, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    tol = ((k + 127) // 128 + 32) * 2.0 ** -23 * mag
    tol = tol + HALF[dt] * (np.abs(want) + tol)
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.max(np.abs(got - want) / tol):.3g} of the tolerance"


@pytest.mark.parametrize("rows", (3, 40, 300))
def test_linear_not_finite(rows):
    """A NaN scale or element takes its own row or column, and nothing else."""
    k, d = 392, 264
    note(f"linear with NaN, {rows} rows")
    for fmt in (R.E4M3, R.E2M1):
        xq, xs = R.quantize(rand(1, rows, k), fmt)
        wq, ws = R.quantize(rand(2, d, k), R.E2M1)
        xs[1, 3], ws[5, 12] = 255, 255
        if fmt == R.E4M3:
            xq[2, 7] = 0x7F
        h = make_weight(d, k, wq, ws)
        try:
            got = linear(h, xq, xs, fmt, rows, d, F32)
        finally:
            lb.lora_mx_weight_destroy(h)
        want = np.zeros((rows, d), bool)
        want[1], want[:, 5] = True, True
        if fmt == R.E4M3:
            want[2] = True
        np.testing.assert_array_equal(np.isnan(got), want)


def test_linear_extreme_scales():
    """Blocks at both ends of the scale range: 2^-127 and 2^127."""
    note("linear extreme scales")
    rows, k, d = 20, 64, 16
    x, w = np.ones((rows, k)), np.ones((d, k))
    xq, wq = R.pack(R.codes_under(x, np.full((rows, 2), 127, np.uint8), R.E4M3), R.E4M3), \
        R.pack(R.codes_under(w, np.full((d, 2), 127, np.uint8), R.E2M1), R.E2M1)
    for a, b in ((0, 254), (254, 0), (0, 127), (10, 130), (254, 127)):
        xs, ws = R.pad_scales(np.full((rows, 2), a, np.uint8), k), R.pad_scales(np.full((d, 2), b, np.uint8), k)
        h = make_weight(d, k, wq, ws)
        try:
            got = linear(h, xq, xs, R.E4M3, rows, d, F32)
        finally:
            lb.lora_mx_weight_destroy(h)
        e = a + b - 254 + 6
        want = np.inf if e > 127 else np.ldexp(1.0, e)
        np.testing.assert_array_equal(got, np.full((rows, d), want))


@pytest.mark.parametrize("dt", (BF, F32))
def test_weight_load_agrees_with_packed(dt):
    """A weight quantised on load and the same one quantised by lora_mx_quantize and loaded packed."""
    d, k = 72, 1288
    note("weight load, dense and packed")
    wd, hw = dense(specials(rand(1, d, k)), dt, 8)
    q, s = blocks(d, k, R.E2M1)
    lb.lora_mx_quantize(*held(q, s), R.E2M1, wd.data_ptr(), wd.stride(0), dt, d, k, stream())
    xq, xs = R.quantize(rand(2, 20, k), R.E4M3)
    got = []
    for load in (lambda w: lb.lora_mx_weight_load(w, wd.data_ptr(), wd.stride(0), dt, stream()),
                 lambda w: lb.lora_mx_weight_load_packed(w, *held(q, s), stream())):
        w = lb.lora_mx_weight_create(d, k)
        with pytest.raises(lb.LoraError) as e:
            lb.lora_mx_linear(w, P_.data_ptr(), d, F32, *held(q, s), R.E2M1, 1, stream())
        assert e.value.status == lb.LORA_E_EMPTY
        load(w)
        got.append(linear(w, xq, xs, R.E4M3, 20, d, F32))
        lb.lora_mx_weight_destroy(w)
    np.testing.assert_array_equal(got[0], got[1])


P_ = torch.zeros(4096, device=DEV) if torch.cuda.is_available() else None


def test_other_stream_and_graph():
    """norm -> product on a side stream, then captured and replayed between eager work: the same bits each time."""
    rows, k, d = 24, 1032, 264
    note("stream and graph")
    x, _ = dense(rand(1, rows, k), BF)
    w, _ = dense(np.ones((1, k)), BF)
    wq, ws = R.quantize(rand(2, d, k), R.E2M1)
    h = make_weight(d, k, wq, ws)
    q, s = blocks(rows, k, R.E4M3)
    y = torch.zeros(rows, d, dtype=torch.bfloat16, device=DEV)

    def step(st):
        lb.lora_rmsnorm_mx(0, 0, *held(q, s), 0, 0, x.data_ptr(), k, 0, 0, w.data_ptr(), 1e-5, BF, rows, k, st)
        lb.lora_mx_linear(h, y.data_ptr(), d, BF, *held(q, s), R.E4M3, rows, st)

    try:
        step(stream())
        torch.cuda.synchronize()
        want = y.clone()
        side = torch.cuda.Stream()
        y.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            step(stream())
        side.synchronize()
        assert torch.equal(y, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(stream())
        for i in range(4):
            y.zero_()
            q.fill_(i)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want), f"replay {i}"
        x.mul_(-1)   # the graph reads its inputs anew
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, -want)
    finally:
        torch.cuda.synchronize()
        lb.lora_mx_weight_destroy(h)


def test_far_offsets():
    """A matrix whose last row starts past 2^32 bytes."""
    rows, k, ld = 3, 264, 1 << 31
    note("far offsets")
    x = torch.zeros(2 * ld + k, dtype=torch.bfloat16, device=DEV)   # 8.6 GB
    v = rand(5, rows, k)
    for i in range(rows):
        x[i * ld:i * ld + k] = torch.from_numpy(v[i]).to(DEV).bfloat16()
    hx = torch.stack([x[i * ld:i * ld + k] for i in range(rows)]).double().cpu().numpy()
    q, s = blocks(rows, k, R.E2M1)
    lb.lora_mx_quantize(*held(q, s), R.E2M1, x.data_ptr(), ld, BF, rows, k, stream())
    want_q, want_s = R.quantize(hx, R.E2M1)
    np.testing.assert_array_equal(q.cpu().numpy()[:rows], want_q)
    np.testing.assert_array_equal(s.cpu().numpy()[:rows], want_s)
    wq, ws = R.quantize(rand(6, 16, k), R.E2M1)
    h = make_weight(16, k, wq, ws)
    try:
        lb.lora_mx_linear(h, x.data_ptr(), ld, BF, *held(q, s), R.E2M1, rows, stream())
        y = torch.stack([x[i * ld:i * ld + 16] for i in range(rows)]).double().cpu().numpy()
        near = linear(h, want_q, want_s, R.E2M1, rows, 16, BF)
        np.testing.assert_array_equal(y, near)
    finally:
        lb.lora_mx_weight_destroy(h)


def test_swiglu_far_and_infinite_gates():
    """Gates where exp overflows or vanishes, infinities and NaN: the formula's value in fp32's range."""
    gates = [0.0, -0.0, 1e-30, -1e-30, 60.0, -60.0, 87.0, -87.0, -88.5, -100.0, 200.0, 1e30, -1e30, np.inf, -np.inf, np.nan]
    ups = [1.0, -2.5, 1e30, 1e-30]
    n, f = len(ups), len(gates)
    x, hx = dense(np.concatenate([np.tile(gates, (n, 1)), np.repeat(np.array(ups)[:, None], f, 1)], 1), F32)
    out = torch.empty(n, f, dtype=torch.float32, device=DEV)
    note("swiglu far gates")
    lb.lora_swiglu_mx(out.data_ptr(), f, 0, 0, 0, 0, x.data_ptr(), 2 * f, F32, n, f, stream())
    got = out.double().cpu().numpy()
    g, u = hx[:, :f], hx[:, f:]
    with np.errstate(all="ignore"):
        ex = g / (1 + np.exp(-g)) * u
        ex = np.where(np.abs(ex) > np.finfo(np.float32).max, np.copysign(np.inf, ex), ex)
        far = (g < -88.73) & np.isfinite(g)   # fp32's exp(-g) overflows past 88.73, and the quotient is 0
        # 16 u of the value, and one subnormal step of each of the two products under 2^-126
        ok = np.abs(got - ex) <= 16 * 2.0 ** -24 * np.abs(ex) + 2.0 ** -149 * (1 + np.abs(u))
    ok |= (got == ex) | (np.isnan(got) & np.isnan(ex))
    ok[far] = got[far] == 0
    assert ok.all(), np.argwhere(~ok).tolist()


@pytest.mark.parametrize("dt", (BF, F32))
def test_swiglu_is_near_the_operations_one_by_one(dt):
    """Against fp32 operations in turn: under one step of fp32, and so (bf16) the same or the neighbouring value."""
    n, f = 64, 4096
    x, _ = dense(rand(23, n, 2 * f, 1.0), dt)
    out = torch.empty(n, f, dtype=TD[dt], device=DEV)
    note("swiglu against fp32 operations")
    lb.lora_swiglu_mx(out.data_ptr(), f, 0, 0, 0, 0, x.data_ptr(), 2 * f, dt, n, f, stream())
    g, u = x[:, :f].float().cpu(), x[:, f:2 * f].float().cpu()
    want = (g / (1 + torch.exp(-g)) * u).to(TD[dt]).double()
    got = out.double().cpu()
    # exp within 2^-23 on either side; sum, quotient and product half a step each on both sides: 2 + 3 steps of 2^-23
    assert ((got - want).abs() <= (5 * 2.0 ** -23 + (2.0 ** -7 if dt == BF else 0)) * want.abs() + 2.0 ** -126).all()


def test_rmsnorm_codes_beside_a_border():
    """Values within 2^-26 of the middle of two codes: fp32's nearest is the middle itself, the codes still fall right.

    h is near 2^-30, so mean h^2 + 1 is 1 in 64 bits and n = h w.  With a = 2^-9, (1 + a)(1 - a + a^2) = 1 + 2^-27, and with
    b = 2^-13, (1 + b)(1 - b) = 1 - 2^-26.  The middles are odd sixteenths; every factor has at most 23 bits.
    """
    a, b, k = 2.0 ** -9, 2.0 ** -13, 264
    pairs = [(2.0 ** -30 * up * sign, m / 16 * rest) for m in (17, 19, 21, 23, 25, 27) for sign in (1, -1)
             for up, rest in ((1 + a, 1 - a + a * a), (1 + b, 1 - b))]
    hv, wv = np.resize(np.array(pairs), (k, 2)).T
    x, hx = dense(hv[None], F32)
    w, hw = dense(wv[None], F32)
    assert (hx == hv).all() and (hw == wv).all()
    exact = hx * hw   # at most 46 bits
    middle = exact.astype(np.float32).astype(np.float64)
    assert (np.abs(middle) * 2.0 ** 34 % 2 == 1).all() and (middle != exact).all()
    q, s = blocks(1, k, R.E4M3)
    note("rmsnorm beside a border")
    lb.lora_rmsnorm_mx(0, 0, *held(q, s), 0, 0, x.data_ptr(), k, 0, 0, w.data_ptr(), 1.0, F32, 1, k, stream())
    check_blocks(q.cpu().numpy(), s.cpu().numpy(), exact, 0.0, k)


def test_rmsnorm_weights_not_finite():
    """h inv w with an infinite or NaN weight: the product's value, and blocks of NaN around it."""
    k = 264
    x, hx = dense(np.where(np.arange(k) % 2, 1.0, -1.0)[None], F32)   # inv is 1
    wv = np.ones((1, k))
    wv[0, [0, 1, 40, 77]] = np.inf, np.inf, -np.inf, np.nan
    w, hw = dense(wv, F32)
    out = torch.empty_like(x)
    q, s = blocks(1, k, R.E4M3)
    note("rmsnorm weights not finite")
    lb.lora_rmsnorm_mx(out.data_ptr(), k, *held(q, s), 0, 0, x.data_ptr(), k, 0, 0, w.data_ptr(), 0.0, F32, 1, k, stream())
    np.testing.assert_array_equal(out.double().cpu().numpy(), hx * hw)
    gs = s.cpu().numpy()[0, :9]
    assert (gs[:3] == 255).all() and (gs[3:] == 127 - 8).all()


def test_rmsnorm_tiny_and_huge_rows():
    """Rows whose mean square is far from one: the root's scaling, and squares past the range (infinite mean: zeros)."""
    rows, k = 4, 256
    g = np.random.default_rng(11)
    v = g.standard_normal((rows, k)) * np.array([1e-16, 1e-18, 1e15, 1e25])[:, None]
    x, hx = dense(v, F32)
    w, hw = dense(np.ones((1, k)), F32)
    out = torch.empty_like(x)
    note("rmsnorm tiny and huge rows")
    lb.lora_rmsnorm_mx(out.data_ptr(), k, 0, 0, 0, 0, 0, 0, x.data_ptr(), k, 0, 0, w.data_ptr(), 0.0, F32, rows, k, stream())
    got = out.double().cpu().numpy()
    _, en = R.norm(hx, None, hw, 0.0)
    # squares of 1e-18 and below round to 2^-149: half of that on each of k / 2 or more terms of mean 1e-36
    check_dense(got[:1], en[:1], F32, 2.0 ** -18, "tiny")
    check_dense(got[1:2], en[1:2], F32, 2.0 ** -12, "tinier")
    check_dense(got[2:3], en[2:3], F32, 2.0 ** -18, "huge")
    assert (got[3] == 0).all()
