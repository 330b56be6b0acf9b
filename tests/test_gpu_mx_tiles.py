"""Every kernel that the microscaled product's launcher chooses between (256 CUs), on inputs that need all of it.

Tolerances: none where sums are exact in fp32 in any order; elsewhere, as the product's own tests, each matrix
instruction (one per 128 k) and each joining of partial sums (under 32) rounds by 2^-23 of the summed magnitudes at
most, and the output is rounded once.
"""
import numpy as np
import pytest
import torch

import mx_cases as C
import mx_reference as R
import test_gpu_mx as T
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb

pytestmark = pytest.mark.gpu

BF, F32 = lb.LORA_BF16, lb.LORA_F32

# direct kernels 16x16, 16x32, 16x32, 16x64, 32x64; then tiles of 64x64 (twice), 64x128 in sets, 64x128, 64x128 or (4 bits)
# 128x128, 128x256 or 256x256
SHAPES = [(9, 520, 72)] + [s for s in T.LINEAR_TILES if s[0] != 7] + [(7, 264, 16000)]


def ones(rows, k):
    return np.full((rows, -(-k // 32)), 127, np.uint8)


def packed(v, fmt):
    return R.pack(R.codes_under(v, ones(*v.shape), fmt), fmt)


def both_types(rows, k, d, fmt, xq, xs, wq, ws, check):
    """check(values got, dtype) for both outputs of one product."""
    h = T.make_weight(d, k, wq, ws, pad=16)
    try:
        for dt in (F32, BF):
            check(T.linear(h, xq, xs, fmt, rows, d, dt, pad=8), dt)
    finally:
        lb.lora_mx_weight_destroy(h)


def exactly(want):
    def check(got, dt):
        np.testing.assert_array_equal(got, want if dt == F32 else R.bf16(want))
    return check


@pytest.mark.parametrize("rows,k,d", SHAPES)
def test_products_that_need_the_split(rows, k, d):
    """448 * 6 beside 2^-9 * 0.5 among eight neighbouring k: no term of an e4m3 product may be dropped."""
    note(f"linear wide products {rows}x{k}x{d}")
    x, w = C.wide_products(rows, k, d, rows + d)
    g = np.random.default_rng(rows)
    sx, sw = g.integers(120, 134, (rows, 1)), g.integers(120, 134, (d, 1))   # one power of two a row moves no bit
    want = np.ldexp(x @ w.T, sx + sw.T - 254)
    blocks = -(-k // 32)
    both_types(rows, k, d, R.E4M3, packed(x, R.E4M3), R.pad_scales(np.repeat(sx, blocks, 1).astype(np.uint8), k),
               packed(w, R.E2M1), R.pad_scales(np.repeat(sw, blocks, 1).astype(np.uint8), k), exactly(want))


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("rows,k,d", SHAPES)
def test_far_block_scales(rows, k, d, fmt):
    """Blocks of X around 2^-100 .. 2^100 whose W blocks bring them back: whole numbers, every bit right."""
    note(f"linear far scales {rows}x{k}x{d} format {fmt}")
    g = np.random.default_rng(k + d)
    x = g.choice([-2.0, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5, 3.0], (rows, k))
    w = g.choice([-6.0, -3.0, -1.0, 0.0, 0.5, 1.0, 2.0, 4.0], (d, k))
    far = g.integers(20, 234, (1, -(-k // 32)))
    sx = (far + g.integers(0, 2, (rows, far.shape[1]))).astype(np.uint8)
    sw = (254 - far + g.integers(0, 2, (d, far.shape[1]))).astype(np.uint8)
    xq, wq, xs, ws = packed(x, fmt), packed(w, R.E2M1), R.pad_scales(sx, k), R.pad_scales(sw, k)
    want = R.values(xq, xs, fmt, k) @ R.values(wq, ws, R.E2M1, k).T
    assert np.abs(want).max() < 2 ** 20   # multiples of 1/4
    both_types(rows, k, d, fmt, xq, xs, wq, ws, exactly(want))


@pytest.mark.parametrize("a,b", ((0, 254), (254, 0), (0, 140), (254, 100), (254, 127)))
@pytest.mark.parametrize("rows,k,d", [s for s in SHAPES if s[0] in (9, 70, 256, 500, 1000, 8190)])
def test_extreme_scales(rows, k, d, a, b):
    """Both ends of the scale range: 2^-127 and 2^127, and sums past fp32's largest."""
    note(f"linear extreme scales {rows}x{k}x{d} {a} {b}")
    e = a + b - 254
    want = np.inf if e + np.log2(k) >= 128 else np.ldexp(float(k), e)
    full = [R.pad_scales(np.full((n, -(-k // 32)), s, np.uint8), k) for n, s in ((rows, a), (d, b))]
    for fmt in (R.E4M3, R.E2M1):
        both_types(rows, k, d, fmt, packed(np.ones((rows, k)), fmt), full[0], packed(np.ones((d, k)), R.E2M1), full[1],
                   exactly(np.full((rows, d), want)))


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("rows,k,d", SHAPES)
def test_not_finite(rows, k, d, fmt):
    """A NaN scale or element takes its own row or column; every other output keeps its bits."""
    note(f"linear with NaN {rows}x{k}x{d} format {fmt}")
    xq, xs = R.quantize(T.rand(1, rows, k), fmt)
    wq, ws = R.quantize(T.rand(2, d, k), R.E2M1)
    clean = {}
    both_types(rows, k, d, fmt, xq, xs, wq, ws, lambda got, dt: clean.update({dt: got}))
    last = -(-k // 32) - 1
    bad_rows, bad_cols = [1, rows - 1], [5, d - 1]
    xs[1, 3], xs[rows - 1, last], ws[5, last], ws[d - 1, 0] = 255, 255, 255, 255
    if fmt == R.E4M3:
        xq[2, 7], xq[4, k - 1] = 0x7F, 0xFF
        bad_rows += [2, 4]

    def check(got, dt):
        want = clean[dt].copy()
        assert np.isfinite(want).all()
        want[bad_rows], want[:, bad_cols] = np.nan, np.nan
        np.testing.assert_array_equal(got, want)
    both_types(rows, k, d, fmt, xq, xs, wq, ws, check)


@pytest.mark.parametrize("fmt", (R.E4M3, R.E2M1))
@pytest.mark.parametrize("rows,k,d", SHAPES)
def test_hidden_states(rows, k, d, fmt):
    note(f"linear hidden states {rows}x{k}x{d} format {fmt}")
    xq, xs = R.quantize(T.rand(rows, rows, k), fmt)
    wq, ws = R.quantize(0.02 * T.rand(d, d, k, 0.3), R.E2M1)
    xv, wv = R.values(xq, xs, fmt, k), R.values(wq, ws, R.E2M1, k)
    want, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    sums = ((k + 127) // 128 + 32) * 2.0 ** -23 * mag

    def check(got, dt):
        bad = np.abs(got - want) > sums + T.HALF[dt] * (np.abs(want) + sums)
        assert not bad.any(), f"{bad.sum()} of {bad.size}"
    both_types(rows, k, d, fmt, xq, xs, wq, ws, check)


def test_shapes_reach_every_kernel():
    """SHAPES is for a card of 256 CUs."""
    assert torch.cuda.get_device_properties(0).multi_processor_count == 256
