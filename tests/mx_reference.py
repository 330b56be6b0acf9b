"""Plain 64-bit forms of the microscaled operators (numpy), from their definitions:
blocks of 32 along k, a power of two per block, elements e4m3 or e2m1."""
from __future__ import annotations

import numpy as np

from rank_adapter_gemm_lora_amd import binding as lb

E4M3, E2M1 = lb.LORA_MX_E4M3, lb.LORA_MX_E2M1
EMAX = {E4M3: 8, E2M1: 2}


def grid(fmt):
    """Values of codes 0 .. largest, ascending (the code is the index)."""
    if fmt == E2M1:
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    e, m = np.arange(127) >> 3, np.arange(127) & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def block_scales(v, fmt):
    """Scale bytes [rows, blocks] of values [rows, k]."""
    rows, k = v.shape
    b = np.zeros((rows, -(-k // 32) * 32))
    b[:, :k] = v
    b = np.abs(b.reshape(rows, -1, 32))
    out = np.zeros(b.shape[:2], np.uint8)
    for i in np.ndindex(*out.shape):
        if not np.isfinite(b[i]).all():
            out[i] = 255
        elif b[i].max() > 0:
            out[i] = max(0, int(np.frexp(b[i].max())[1]) - 1 - EMAX[fmt] + 127)
    return out


def codes_under(v, scales, fmt):
    """Codes [rows, k] of values under given scale bytes: nearest, ties to the even code, saturating."""
    rows, k = v.shape
    s = np.repeat(scales, 32, axis=1)[:, :k].astype(int)
    bad = s == 255
    u = np.where(bad, 0.0, np.ldexp(np.where(bad, 0.0, np.abs(v)), 127 - s))
    g = grid(fmt)
    mid = (g[1:] + g[:-1]) / 2
    i = np.searchsorted(mid, u)
    tie = (i < len(mid)) & (u == mid[np.minimum(i, len(mid) - 1)]) & (i % 2 == 1)
    i = i + tie
    sign = np.where(bad, False, np.signbit(v))
    return (i + np.where(sign, 128 if fmt == E4M3 else 8, 0)).astype(np.uint8)


def pack(codes, fmt):
    """Codes [rows, k] -> rows of lora_mx_code_bytes(k) bytes."""
    rows, k = codes.shape
    full = np.zeros((rows, (k + 127) // 128 * 128), np.uint8)
    full[:, :k] = codes
    return full if fmt == E4M3 else (full[:, 0::2] | full[:, 1::2] << 4)


def pad_scales(s, k):
    full = np.zeros((s.shape[0], lb.lora_mx_scale_bytes(k)), np.uint8)
    full[:, :s.shape[1]] = s
    return full


def quantize(v, fmt):
    """(packed codes, padded scales) of values [rows, k]."""
    s = block_scales(v, fmt)
    return pack(codes_under(v, s, fmt), fmt), pad_scales(s, v.shape[1])


def unpack(q, fmt, k):
    if fmt == E4M3:
        return q[:, :k]
    c = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    c[:, 0::2], c[:, 1::2] = q & 15, q >> 4
    return c[:, :k]


def values(q, s, fmt, k):
    """What packed codes and scales stand for, [rows, k] in float64."""
    c = unpack(q, fmt, k).astype(int)
    half = 128 if fmt == E4M3 else 8
    g = np.append(grid(fmt), np.nan) if fmt == E4M3 else grid(fmt)
    v = g[c % half] * np.where(c >= half, -1.0, 1.0)
    e = np.repeat(s.astype(int), 32, axis=1)[:, :k]
    return np.where(e == 255, np.nan, np.ldexp(v, np.where(e == 255, 0, e - 127)))


def bf16(v):
    """Float values -> the nearest bf16 values (as float64), ties to even."""
    import torch
    return torch.from_numpy(np.asarray(v, np.float32)).bfloat16().double().numpy()


def norm(x, r, w, eps):
    h = x if r is None else x + r
    return h, h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w


def swiglu(gu):
    f = gu.shape[1] // 2
    g, u = gu[:, :f], gu[:, f:]
    return g / (1 + np.exp(-g)) * u
