"""lora_block_norm_mx on the GPU against its formula in 64 bits.

Tolerances, from the roundings counted before the first run: the kernel and the reference both compute in 64 bits
(under 200 roundings of 2^-53 each on the way to n, the sum's included, far below 2^-40 of the value where h is no
difference of near numbers; where residual and block nearly cancel, the same against the larger of the two).  An
output is that value rounded once: half a step, 2^-8 / 2^-24 of it.  Codes lie between those of the exact values
moved down and up by 2^-40.
"""
import numpy as np
import pytest
import torch

import mx_reference as R
from gpu_helpers import note
from rank_adapter_gemm_lora_amd import binding as lb
from test_gpu_mx import BF, DEV, F32, FILL, HALF, blocks, check_blocks, dense, held, rand, stream

pytestmark = pytest.mark.gpu

EPS, SCALE = 1e-5, 0.75
FINE = 2.0 ** -40


def reference(y, r, post, gate, scale, pre, eps):
    def rms(v):
        return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    a = y if post is None else rms(y) * post
    m = scale * a * (1.0 if gate is None else gate)
    h = m if r is None else r + m
    size = np.abs(m) if r is None else np.maximum(np.abs(m), np.abs(r))
    return h, None if pre is None else rms(h) * pre, size


def near(got, want, dt, slack, what):
    """got is want rounded once, want known within slack."""
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= HALF[dt] * np.abs(want) + 2 * slack + 2.0 ** -133)
    bad &= ~(np.isnan(got) & np.isnan(want)) & ~(got == want)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}"


def call(rows, k, dt, y, r, post, gate, ldg, pre, out, h, q, s, scale=SCALE, eps=EPS):
    def at(t):
        return 0 if t is None else t.data_ptr()

    def ld(t):
        return 0 if t is None else t.stride(0)
    qs = (0, 0, 0, 0) if q is None else held(q, s)
    lb.lora_block_norm_mx(at(out), ld(out), *qs, at(h), ld(h), at(y), ld(y), at(r), ld(r), at(post), at(gate), ldg, scale,
                          at(pre), eps, dt, rows, k, stream())


SHAPES = [(1, 8), (3, 40), (2, 136), (17, 512), (5, 520), (33, 1032), (4, 2056), (65, 4096), (3, 4104), (2, 8200), (2, 16392),
          (1, 32768)]


@pytest.mark.parametrize("dt", (BF, F32))
@pytest.mark.parametrize("rows,k", SHAPES)
@pytest.mark.parametrize("post,gate,residual", [(True, "none", True), (True, "row", True), (False, "channel", True),
                                                (True, "channel", False), (False, "none", False)])
def test_block_norm(rows, k, post, gate, residual, dt):
    note(f"block norm {rows}x{k} dtype {dt} post {post} gate {gate} residual {residual}")
    v = rand(rows + k, rows, k)
    if rows > 2:
        v[1] = 0
    y, hy = dense(v, dt, 8)
    r, hr = dense(rand(3 * rows + k, rows, k), dt, 16)
    g, hg = dense(rand(5 * rows + k, 1 if gate == "channel" else rows, k, 0.3), dt, 24)
    wp, hp = dense(0.5 + 0.2 * rand(6, 1, k, 0.0), dt)
    wn, hn = dense(1 + 0.2 * rand(7, 1, k, 0.0), dt)
    out = torch.full((rows + 1, k + 8), 7.0, dtype=y.dtype, device=DEV)
    h = torch.full((rows + 1, k + 16), 7.0, dtype=y.dtype, device=DEV)
    q, s = blocks(rows, k, R.E4M3, 16)
    call(rows, k, dt, y, r if residual else None, wp if post else None, None if gate == "none" else g,
         g.stride(0) if gate == "row" else 0, wn, out, h, q, s)
    eps = float(np.float32(EPS))
    eh, en, size = reference(hy, hr if residual else None, hp if post else None, None if gate == "none" else hg, SCALE, hn, eps)
    gh, gn = h.double().cpu().numpy(), out.double().cpu().numpy()
    near(gh[:rows, :k], eh, dt, FINE * size, "h")
    with np.errstate(divide="ignore", invalid="ignore"):
        slack = np.where(eh != 0, FINE * size * np.abs(en / eh), FINE * np.abs(size * hn / np.sqrt((eh * eh).mean(-1, keepdims=True) + eps)))
    near(gn[:rows, :k], en, dt, slack, "out")
    assert (gh[rows:] == 7).all() and (gh[:, k:] == 7).all() and (gn[rows:] == 7).all() and (gn[:, k:] == 7).all()
    gq, gs = q.cpu().numpy(), s.cpu().numpy()
    check_blocks(gq, gs, en, FINE, k)
    assert (gq[rows:] == FILL).all() and (gq[:, lb.lora_mx_code_bytes(k, R.E4M3):] == FILL).all()
    assert (gs[rows:] == FILL).all() and (gs[:, lb.lora_mx_scale_bytes(k):] == FILL).all()


@pytest.mark.parametrize("dt", (BF, F32))
def test_block_norm_in_place_and_outputs_left_out(dt):
    rows, k = 5, 264
    y, hy = dense(rand(1, rows, k), dt)
    r, hr = dense(rand(2, rows, k), dt)
    wp, hp = dense(rand(3, 1, k, 0.0), dt)
    wn, hn = dense(rand(4, 1, k, 0.0), dt)
    note(f"block norm in place dtype {dt}")
    eh, en, size = reference(hy, hr, hp, None, SCALE, hn, float(np.float32(EPS)))
    y1, r1 = y.clone(), r.clone()
    call(rows, k, dt, y1, r1, wp, None, 0, wn, y1, r1, None, None)   # h over the residual, n over y
    near(r1.double().cpu().numpy(), eh, dt, FINE * size, "h")
    full = y1.clone()
    y2 = y.clone()
    call(rows, k, dt, y2, r, wp, None, 0, None, None, y2, None, None)   # no second norm: h alone, over y
    assert torch.equal(y2, r1)
    q, s = blocks(rows, k, R.E4M3)
    call(rows, k, dt, y, r, wp, None, 0, wn, None, None, q, s)   # blocks alone
    check_blocks(q.cpu().numpy(), s.cpu().numpy(), en, FINE, k)
    out = torch.empty_like(y)
    call(rows, k, dt, y, r, wp, None, 0, wn, out, None, None, None)   # n alone
    assert torch.equal(out, full)


@pytest.mark.parametrize("dt", (BF, F32))
def test_block_norm_special_rows(dt):
    """Zeros under eps 0, NaN, infinities, rows at both ends of the range."""
    rows, k = 7, 136
    v = rand(9, rows, k, 0.0)
    v[0] = 0
    v[1, 5], v[2, 9] = np.nan, np.inf
    v[3] *= 1e30
    v[4] *= 1e-30
    y, hy = dense(v, dt)
    r, hr = dense(np.where(np.arange(rows)[:, None] == 5, 1e30, 0.0) * np.ones((rows, k)), dt)
    w, hw = dense(np.ones((1, k)), dt)
    out, h = torch.empty_like(y), torch.empty_like(y)
    q, s = blocks(rows, k, R.E4M3)
    note(f"block norm special rows dtype {dt}")
    call(rows, k, dt, y, r, w, None, 0, w, out, h, q, s, scale=1.0, eps=0.0)
    gh, gn, gs = h.double().cpu().numpy(), out.double().cpu().numpy(), s.cpu().numpy()
    assert np.isnan(gh[0]).all() and np.isnan(gh[1]).all()   # 0 / 0; a NaN takes its row
    assert np.isnan(gh[2, 9]) and (gh[2, :9] == 0).all()     # inf / inf, the rest over inf
    assert np.isnan(gn[:3]).all() and (gs[:3, :5] == 255).all() and not q.cpu().numpy()[:3].any()
    eh, en, size = reference(hy[3:], hr[3:], hw, None, 1.0, hw, 0.0)
    near(gh[3:], eh, dt, FINE * size, "h")
    near(gn[3:], en, dt, FINE * np.abs(en), "out")


def test_block_norm_another_stream_and_replays():
    rows, k = 40, 4096
    y, _ = dense(rand(1, rows, k), BF)
    r, _ = dense(rand(2, rows, k), BF)
    w, _ = dense(rand(3, 1, k, 0.0), BF)
    out, h = torch.empty_like(y), torch.empty_like(y)
    q, s = blocks(rows, k, R.E4M3)
    args = (rows, k, BF, y, r, w, w, 0, w, out, h, q, s)
    note("block norm captured")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*args)
    for i in range(3):
        y.copy_((y.float() * 1.5 + i).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (out, h, q, s)]
        call(*args)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, h, q, s))), f"replay {i}"
