"""What is timed of the microscaled (MX) operators, and their plain forms.

The base projections that the adapters' deltas are added to, with 4-bit weights
and 8- or 4-bit activations in blocks of 32 along k that share one power of two
(OCP microscaling: elements e4m3 or e2m1, scales e8m0):

  norm      h = x + residual; n = h * rsqrt(mean(h^2) + eps) * w; n again in e4m3 blocks
  swiglu    a = silu(g) * u; a again in e4m3 blocks
  quantize  a matrix in e4m3 or e2m1 blocks
  linear    y = A W^T of an activation in e4m3 or e2m1 blocks and a weight in e2m1 blocks

An output in blocks is returned as the values that it stands for (element times
scale).  Where ``own`` is true, run() makes the library's calls instead.
"""
import math

import torch

own = False

DEV = "cuda:0"
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# exponent of the largest binade, smallest normal exponent, fraction bits, largest value
FORMATS = {"e4m3": (8, -6, 3, 448.0), "e2m1": (2, 0, 1, 6.0)}


def listed():
    return [
        # one request decoding alone: latency
        {"name": "norm_1x4096", "op": "norm", "rows": 1, "k": 4096, "dtype": "bf16", "residual": True},
        # a decode batch ahead of the attention projections
        {"name": "norm_256x4096", "op": "norm", "rows": 256, "k": 4096, "dtype": "bf16", "residual": True},
        # a prefill batch, rows of many prompts one after the other
        {"name": "norm_35422x4096", "op": "norm", "rows": 35422, "k": 4096, "dtype": "bf16", "residual": True},
        # the MLP's activation of a few decoding requests, kept in fp32
        {"name": "swiglu_16x14336_f32", "op": "swiglu", "rows": 16, "k": 14336, "dtype": "f32"},
        # the same of a mixed batch
        {"name": "swiglu_512x14336", "op": "swiglu", "rows": 512, "k": 14336, "dtype": "bf16"},
        # a weight of the MLP turned into 4 bits
        {"name": "quantize_14336x4096_e2m1", "op": "quantize", "rows": 14336, "k": 4096, "dtype": "bf16", "fmt": "e2m1"},
        # an attention output on its way into its projection: odd rows, a last block that is not whole
        {"name": "quantize_1023x4104_e4m3", "op": "quantize", "rows": 1023, "k": 4104, "dtype": "f32", "fmt": "e4m3"},
        # q/k/v of one decoding request
        {"name": "linear_1x4096x6144", "op": "linear", "rows": 1, "k": 4096, "d": 6144, "dtype": "bf16", "fmt": "e4m3"},
        # q of a decode batch
        {"name": "linear_256x4096x4096", "op": "linear", "rows": 256, "k": 4096, "d": 4096, "dtype": "bf16", "fmt": "e4m3"},
        # the MLP's down projection, activations in 4 bits too, summed on in fp32 by the caller
        {"name": "linear_512x14336x4096_e2m1", "op": "linear", "rows": 512, "k": 14336, "d": 4096, "dtype": "f32", "fmt": "e2m1"},
        # a wide projection under a thousand rows of as many requests
        {"name": "linear_1024x8192x28672", "op": "linear", "rows": 1024, "k": 8192, "d": 28672, "dtype": "bf16", "fmt": "e4m3"},
        # q/k/v of a prefill batch
        {"name": "linear_35422x4096x6144", "op": "linear", "rows": 35422, "k": 4096, "d": 6144, "dtype": "bf16", "fmt": "e4m3"},
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def _eights(rng, lo, hi):
    return max(8, _log(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(["norm", "swiglu", "quantize", "linear", "linear", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    case = {"op": op, "dtype": dtype}
    if op == "linear":
        k, d = _eights(rng, 64, 14336), _eights(rng, 64, 28672)
        most = min(35422, (1 << 39) // (k * d))
        return case | {"rows": _log(rng, 1, most), "k": k, "d": d, "fmt": rng.choice(["e4m3", "e4m3", "e2m1"])}
    k = _eights(rng, 64, 28672 if op == "swiglu" else 14336)
    case |= {"rows": _log(rng, 1, min(35422, (1 << 26) // k)), "k": k}
    if op == "norm":
        case["residual"] = rng.random() < 0.8
    if op == "quantize":
        case["fmt"] = rng.choice(["e4m3", "e2m1"])
    return case


# ------------------------------------------------------------- plain forms

def _exp2(e, dtype):
    return torch.ldexp(torch.ones((), dtype=dtype, device=e.device), e)


def _blocks(v):
    """[rows, k] -> [rows, blocks, 32], the last block filled with zeros."""
    rows, k = v.shape
    return torch.nn.functional.pad(v, (0, -k % 32)).view(rows, -1, 32)


def _parts(v, fmt):
    """(elements [rows, blocks, 32], exponent of each block's scale [rows, blocks, 1])."""
    top, low, bits, most = FORMATS[fmt]
    b = _blocks(v)
    peak = b.abs().amax(-1, keepdim=True)
    e = torch.where(peak > 0, torch.frexp(peak)[1] - 1 - top, -127).clamp(-127, 127)
    u = torch.ldexp(b, -e)
    ulp = _exp2((torch.frexp(u)[1] - 1).clamp(min=low) - bits, v.dtype)
    return (torch.round(u / ulp) * ulp).clamp(-most, most), e


def _values(v, fmt):
    """What [rows, k] stands for once it is held in blocks."""
    q, e = _parts(v, fmt)
    return torch.ldexp(q, e).flatten(1)[:, :v.shape[1]]


def _table(fmt, device):
    """The values of all codes of a format, as fp32."""
    top, low, bits, most = FORMATS[fmt]
    n = 256 if fmt == "e4m3" else 16
    c = torch.arange(n, device=device)
    sign = torch.where(c >= n // 2, -1.0, 1.0)
    ex, fr = (c % (n // 2)) >> bits, (c & ((1 << bits) - 1)).float()
    bias = 1 - low
    val = torch.where(ex > 0, _exp2(ex - bias, torch.float32) * (1 + fr / (1 << bits)), fr / (1 << bits) * 2.0 ** low)
    if fmt == "e4m3":
        val[127] = val[255] = float("nan")
        sign[127] = 1.0
    return sign * val


def _decode(codes, scales, fmt, k):
    """Held codes and scales -> the values [rows, k] in fp32."""
    if fmt == "e2m1":
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(1)
    v = _table(fmt, codes.device)[codes.int()]
    n = v.shape[1] // 32
    return (v.view(len(v), n, 32) * _exp2(scales[:, :n, None].int() - 127, torch.float32)).flatten(1)[:, :k]


# ------------------------------------------------------------- inputs

def _ups(n, m):
    return -(-n // m) * m


def _code_bytes(k, fmt):
    return _ups(k, 128) // (1 if fmt == "e4m3" else 2)


def _scale_bytes(k):
    return _ups(k, 512) // 32


def _held(v, fmt):
    """(codes, scales) as a program holds them: rows of whole 128 elements and 512 elements' scales, zeros past k."""
    rows, k = v.shape
    q, e = _parts(v, fmt)
    q = q.flatten(1)
    if fmt == "e4m3":
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
        c = torch.bucketize(q.abs(), edges).to(torch.uint8) + 8 * torch.signbit(q).to(torch.uint8)
        codes = c[:, 0::2] | (c[:, 1::2] << 4)
    pad = torch.nn.functional.pad
    codes = pad(codes, (0, _code_bytes(k, fmt) - codes.shape[1]))
    scales = (e[:, :, 0] + 127).to(torch.uint8)
    return codes.contiguous(), pad(scales, (0, _scale_bytes(k) - scales.shape[1])).contiguous()


def _hidden(g, rows, k, dtype, size=1.0):
    """Hidden states: normal, with a few channels far larger than the others."""
    ch = torch.exp(0.5 * torch.randn(k, generator=g, device=DEV))
    ch[torch.randint(0, k, (max(1, k // 512),), generator=g, device=DEV)] *= 20
    return (torch.randn(rows, k, generator=g, device=DEV) * (ch * size)).to(dtype)


class _Weight:
    """A weight as the library keeps it, freed with the state that holds it."""

    def __init__(self, d, k, codes, scales):
        from rank_adapter_gemm_lora_amd import binding as lb
        self.lb = lb
        self.at = lb.lora_mx_weight_create(d, k)
        lb.lora_mx_weight_load_packed(self.at, codes.data_ptr(), codes.shape[1], scales.data_ptr(), scales.shape[1], _stream())

    def __del__(self):
        self.lb.lora_mx_weight_destroy(self.at)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rows, k, dt = case["rows"], case["k"], DT[case["dtype"]]
    s = {"case": case}
    if case["op"] == "linear":
        d, fmt = case["d"], case["fmt"]
        x = _hidden(g, rows, k, torch.float32)
        w = torch.randn(d, k, generator=g, device=DEV) * (0.02 * torch.exp(0.3 * torch.randn(d, 1, generator=g, device=DEV)))
        s["q"], s["s"] = _held(x, fmt)
        s["wq"], s["ws"] = _held(w, "e2m1")
        s["y"] = torch.empty(rows, d, dtype=dt, device=DEV)
        if own:
            s["w"] = _Weight(d, k, s["wq"], s["ws"])
        return s
    fmt = case.get("fmt", "e4m3")
    s["q"] = torch.empty(rows, _code_bytes(k, fmt), dtype=torch.uint8, device=DEV)
    s["s"] = torch.empty(rows, _scale_bytes(k), dtype=torch.uint8, device=DEV)
    s["v"] = torch.empty(rows, k, dtype=dt, device=DEV)
    s["out"] = torch.empty(rows, k, dtype=dt, device=DEV)
    if case["op"] == "norm":
        s["x"] = _hidden(g, rows, k, dt)
        s["w"] = (1 + 0.2 * torch.randn(k, generator=g, device=DEV)).to(dt)
        s["r"] = _hidden(g, rows, k, dt, 3.0) if case["residual"] else None
        s["h"] = torch.empty(rows, k, dtype=dt, device=DEV) if case["residual"] else None
    elif case["op"] == "swiglu":
        s["x"] = _hidden(g, rows, 2 * k, dt, 1.5)
    else:
        s["x"] = _hidden(g, rows, k, dt)
    return s


# ------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    c = s["case"]
    dt = DT[c["dtype"]]
    if c["op"] == "linear":
        a = _decode(s["q"], s["s"], c["fmt"], c["k"])
        return (a @ _decode(s["wq"], s["ws"], "e2m1", c["k"]).T).to(dt)
    x = s["x"].float()
    if c["op"] == "quantize":
        return _values(x, c["fmt"]).to(dt)
    if c["op"] == "swiglu":
        g, u = x[:, :c["k"]], x[:, c["k"]:]
        a = g / (1 + torch.exp(-g)) * u
        return {"out": a.to(dt), "held": _values(a, "e4m3").to(dt)}
    h = x if s["r"] is None else x + s["r"].float()
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"].float()
    got = {"out": n.to(dt), "held": _values(n, "e4m3").to(dt)}
    return got if s["r"] is None else got | {"h": h.to(dt)}


def _run_own(s):
    from rank_adapter_gemm_lora_amd import binding as lb
    c, st = s["case"], _stream()
    rows, k = c["rows"], c["k"]
    dt = lb.LORA_BF16 if c["dtype"] == "bf16" else lb.LORA_F32
    fmt = lb.LORA_MX_E2M1 if c.get("fmt") == "e2m1" else lb.LORA_MX_E4M3
    q, sc = s["q"], s["s"]
    held = (q.data_ptr(), q.stride(0), sc.data_ptr(), sc.stride(0))
    if c["op"] == "linear":
        lb.lora_mx_linear(s["w"].at, s["y"].data_ptr(), c["d"], dt, *held, fmt, rows, st)
        return s["y"]
    if c["op"] == "quantize":
        lb.lora_mx_quantize(*held, fmt, s["x"].data_ptr(), k, dt, rows, k, st)
        lb.lora_mx_dequantize(s["v"].data_ptr(), k, dt, *held, fmt, rows, k, st)
        return s["v"]
    if c["op"] == "swiglu":
        lb.lora_swiglu_mx(s["out"].data_ptr(), k, *held, s["x"].data_ptr(), 2 * k, dt, rows, k, st)
        lb.lora_mx_dequantize(s["v"].data_ptr(), k, dt, *held, fmt, rows, k, st)
        return {"out": s["out"], "held": s["v"]}
    r, h = s["r"], s["h"]
    lb.lora_rmsnorm_mx(s["out"].data_ptr(), k, *held, 0 if h is None else h.data_ptr(), k, s["x"].data_ptr(), k,
                       0 if r is None else r.data_ptr(), k, s["w"].data_ptr(), EPS, dt, rows, k, st)
    lb.lora_mx_dequantize(s["v"].data_ptr(), k, dt, *held, fmt, rows, k, st)
    got = {"out": s["out"], "held": s["v"]}
    return got if r is None else got | {"h": h}


# ------------------------------------------------------------- in 64 bits

def _nearest(v, fmt):
    """The values that [rows, k] stands for in blocks, by search among the format's values."""
    top = FORMATS[fmt][0]
    rows, k = v.shape
    n = -(-k // 32)
    b = torch.zeros(rows, n * 32, dtype=torch.float64, device=v.device)
    b[:, :k] = v
    b = b.view(rows, n, 32)
    peak = b.abs().max(-1, keepdim=True).values
    # the binade of the largest: log2 may round up onto a power of two
    lg = torch.floor(torch.log2(peak.clamp(min=2.0 ** -140)))
    lg = lg - (torch.exp2(lg) > peak).double() + (torch.exp2(lg + 1) <= peak).double()
    scale = torch.exp2((lg - top).clamp(-127, 127))
    if fmt == "e4m3":
        grid = torch.arange(127, dtype=torch.uint8, device=v.device).view(torch.float8_e4m3fn).double()
    else:
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)
    u = b.abs() / scale
    mid = (grid[1:] + grid[:-1]) / 2
    i = torch.searchsorted(mid, u)               # a tie goes to the lower one ...
    i = torch.where((i < len(mid)) & (i % 2 == 1) & (u == mid[i.clamp(max=len(mid) - 1)]), i + 1, i)  # ... unless that is odd
    return (grid[i] * torch.sign(b) * scale).reshape(rows, -1)[:, :k]


def _meant(codes, scales, fmt, k):
    """Held codes and scales -> [rows, k] in fp64, from the bits."""
    if fmt == "e4m3":
        v = codes.view(torch.float8_e4m3fn).double()
    else:
        c = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.int32, device=codes.device)
        c[:, 0::2], c[:, 1::2] = codes % 16, codes // 16
        m, ex = c % 2, c // 2 % 4
        v = torch.where(ex == 0, m * 0.5, (1 + m * 0.5) * torch.exp2(ex.double() - 1)) * (1 - 2 * (c // 8)).double()
    p = torch.exp2(scales.double() - 127)
    return (v * p.repeat_interleave(32, dim=1)[:, :v.shape[1]])[:, :k]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    k = c["k"]
    if c["op"] == "linear":
        return torch.matmul(_meant(s["q"], s["s"], c["fmt"], k), _meant(s["wq"], s["ws"], "e2m1", k).t())
    x = s["x"].double()
    if c["op"] == "quantize":
        return _nearest(x, c["fmt"])
    if c["op"] == "swiglu":
        a = x[:, :k] * torch.special.expit(x[:, :k]) * x[:, k:]
        return {"out": a, "held": _nearest(a, "e4m3")}
    h = x if s["r"] is None else x + s["r"].double()
    n = s["w"].double() * h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / k + EPS)
    got = {"out": n, "held": _nearest(n, "e4m3")}
    return got if s["r"] is None else got | {"h": h}


# ------------------------------------------------------------- what a pass needs

def work(case):
    c = case
    rows, k, e = c["rows"], c["k"], 2 if c["dtype"] == "bf16" else 4
    per = {"e4m3": 1.0, "e2m1": 0.5}[c.get("fmt", "e4m3")] + 1 / 32   # bytes an element held in blocks takes
    if c["op"] == "linear":
        d = c["d"]
        return {"bytes": rows * k * per + d * k * (0.5 + 1 / 32) + rows * d * e, "flops": 2 * rows * k * d}
    if c["op"] == "quantize":
        return {"bytes": rows * k * (e + e), "flops": 4 * rows * k}
    if c["op"] == "swiglu":
        return {"bytes": rows * k * (2 * e + e + e), "flops": 10 * rows * k}
    return {"bytes": rows * k * ((5 if c["residual"] else 3) * e) + k * e, "flops": 10 * rows * k}
