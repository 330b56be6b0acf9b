"""What is timed of a mixture layer's operators, and their plain forms.

Next to the base projections in 4 bits (weights in e2m1 blocks, activations in
e4m3 or e2m1 blocks of 32 along k that share one power of two):

  norm    the norms after one block and before the next, with the block's gate and residual scale:
          a = y * rsqrt(mean(y^2) + eps) * w_post; h = residual + scale * gate * a;
          n = h * rsqrt(mean(h^2) + eps) * w_pre; n again in e4m3 blocks
  route   logits -> each row's top_k experts, their weights, and the (row, choice) pairs grouped by expert
  fused   y = act(A W^T + bias) + residual, as values or in e4m3 blocks
  up      for every pair, act(a_row W_e^T + bias_e) of its expert e, in grouped order; gated: silu(g) * u
  down    the pairs' rows through their experts' second weights, and each row's sum of them:
          out = residual + sum_j weight_j * y_j

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
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def listed():
    return [
        # between attention and the MLP of one decoding request: latency
        {"name": "norm_1x4096", "op": "norm", "rows": 1, "k": 4096, "dtype": "bf16", "post": True, "gate": "none"},
        # a prefill batch, gated channel by channel
        {"name": "norm_35422x4096", "op": "norm", "rows": 35422, "k": 4096, "dtype": "bf16", "post": True, "gate": "channel"},
        # a decode batch's routing, a few of its rows padding
        {"name": "route_64x64", "op": "route", "rows": 64, "experts": 64, "top_k": 8, "dtype": "f32", "score": "softmax",
         "masked": True},
        # a prefill batch's routing; bf16 logits bring ties
        {"name": "route_35422x128", "op": "route", "rows": 35422, "experts": 128, "top_k": 8, "dtype": "bf16",
         "score": "sigmoid", "masked": False},
        # q/k/v with bias of one decoding request
        {"name": "fused_1x4096x6144", "op": "fused", "rows": 1, "k": 4096, "d": 6144, "dtype": "bf16", "fmt": "e4m3",
         "bias": True, "act": "none", "residual": False, "held": False},
        # the first product of an MLP, straight into the blocks that the second one reads
        {"name": "fused_512x4096x14336_gelu", "op": "fused", "rows": 512, "k": 4096, "d": 14336, "dtype": "bf16",
         "fmt": "e4m3", "bias": True, "act": "gelu", "residual": False, "held": True},
        # the second product of a prefill batch, onto the residual
        {"name": "fused_16384x14336x4096", "op": "fused", "rows": 16384, "k": 14336, "d": 4096, "dtype": "bf16",
         "fmt": "e4m3", "bias": False, "act": "none", "residual": True, "held": False},
        # one decoding request: every pair its own expert, bound by their weights
        {"name": "up_1", "op": "up", "rows": 1, "experts": 64, "top_k": 8, "k": 4096, "f": 1024, "dtype": "bf16",
         "fmt": "e4m3", "act": "swiglu", "bias": False, "held": True},
        # a small batch of odd sizes through ungated experts, activations in 4 bits
        {"name": "up_199_e2m1_gelu", "op": "up", "rows": 199, "experts": 24, "top_k": 3, "k": 1000, "f": 2056, "dtype": "f32",
         "fmt": "e2m1", "act": "gelu_tanh", "bias": True, "held": False},
        # a prefill batch
        {"name": "up_8192", "op": "up", "rows": 8192, "experts": 64, "top_k": 8, "k": 4096, "f": 1024, "dtype": "bf16",
         "fmt": "e4m3", "act": "swiglu", "bias": False, "held": True},
        # a decode batch
        {"name": "down_256", "op": "down", "rows": 256, "experts": 64, "top_k": 8, "f": 1024, "d": 4096, "dtype": "bf16",
         "fmt": "e4m3", "residual": True},
        # a prefill batch, summed on in fp32
        {"name": "down_8192_f32", "op": "down", "rows": 8192, "experts": 64, "top_k": 8, "f": 1024, "d": 4096, "dtype": "f32",
         "fmt": "e4m3", "residual": True},
    ]


def _log(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def _eights(rng, lo, hi):
    return max(8, _log(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(["norm", "route", "fused", "up", "down"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "norm":
        k = _eights(rng, 64, 14336)
        return case | {"rows": _log(rng, 1, min(35422, (1 << 26) // k)), "k": k, "post": rng.random() < 0.7,
                       "gate": rng.choice(["none", "channel", "row"])}
    if op == "route":
        experts = _log(rng, 2, 256)
        return case | {"rows": _log(rng, 1, min(35422, (1 << 22) // experts)), "experts": experts,
                       "top_k": rng.randint(1, min(8, experts)), "score": rng.choice(["softmax", "softmax", "sigmoid"]),
                       "masked": rng.random() < 0.5}
    case["fmt"] = rng.choice(["e4m3", "e4m3", "e2m1"])
    if op == "fused":
        k, d = _eights(rng, 64, 14336), _eights(rng, 64, 14336)
        return case | {"rows": _log(rng, 1, min(16384, (1 << 38) // (k * d))), "k": k, "d": d, "bias": rng.random() < 0.5,
                       "act": rng.choice(ACTS), "residual": rng.random() < 0.5, "held": rng.random() < 0.4}
    experts = _log(rng, 2, 128)
    top_k = rng.randint(1, min(8, experts))
    wide, f = _eights(rng, 64, 4096), _eights(rng, 32, 2048)
    case |= {"rows": _log(rng, 1, min(8192, 65536 // top_k, (1 << 38) // (wide * f * top_k))), "experts": experts,
             "top_k": top_k, "f": f}
    if op == "down":
        return case | {"d": wide, "residual": rng.random() < 0.7}
    return case | {"k": wide, "act": rng.choice(("swiglu", "swiglu") + ACTS), "bias": rng.random() < 0.3,
                   "held": rng.random() < 0.6}


# ------------------------------------------------------------- plain forms

def _exp2(e, dtype):
    return torch.ldexp(torch.ones((), dtype=dtype, device=e.device), e)


def _parts(v, fmt):
    """(elements [rows, blocks, 32], exponent of each block's scale [rows, blocks, 1])."""
    top, low, bits, most = FORMATS[fmt]
    b = torch.nn.functional.pad(v, (0, -v.shape[1] % 32)).view(len(v), -1, 32)
    peak = b.abs().amax(-1, keepdim=True)
    e = torch.where(peak > 0, torch.frexp(peak)[1] - 1 - top, -127).clamp(-127, 127)
    u = torch.ldexp(b, -e)
    ulp = _exp2((torch.frexp(u)[1] - 1).clamp(min=low) - bits, v.dtype)
    return (torch.round(u / ulp) * ulp).clamp(-most, most), e


def _values(v, fmt="e4m3"):
    """What [rows, k] stands for once it is held in blocks."""
    q, e = _parts(v, fmt)
    return torch.ldexp(q, e).flatten(1)[:, :v.shape[1]]


def _table(fmt, device):
    """The values of all codes of a format, as fp32."""
    top, low, bits, most = FORMATS[fmt]
    n = 256 if fmt == "e4m3" else 16
    c = torch.arange(n, device=device)
    ex, fr = (c % (n // 2)) >> bits, (c & ((1 << bits) - 1)).float() / (1 << bits)
    val = torch.where(ex > 0, _exp2(ex - 1 + low, torch.float32) * (1 + fr), fr * 2.0 ** low)
    if fmt == "e4m3":
        val[127] = val[255] = float("nan")
    return torch.where(c >= n // 2, -1.0, 1.0) * val


def _decode(codes, scales, fmt, k):
    """Held codes and scales -> the values [rows, k] in fp32."""
    if fmt == "e2m1":
        codes = torch.stack((codes & 15, codes >> 4), -1).flatten(1)
    v = _table(fmt, codes.device)[codes.int()]
    n = v.shape[1] // 32
    return (v.view(len(v), n, 32) * _exp2(scales[:, :n, None].int() - 127, torch.float32)).flatten(1)[:, :k]


def _act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))
    if act == "swiglu":
        g, u = v.chunk(2, dim=1)
        return g / (1 + torch.exp(-g)) * u
    return v


# ------------------------------------------------------------- inputs

def _ups(n, m):
    return -(-n // m) * m


def _code_bytes(k, fmt):
    return _ups(k, 128) // (1 if fmt == "e4m3" else 2)


def _scale_bytes(k):
    return _ups(k, 512) // 32


def _held(v, fmt):
    """(codes, scales) as a program holds them: rows of whole 128 elements and 512 elements' scales, zeros past k."""
    k = v.shape[1]
    q, e = _parts(v, fmt)
    q = q.flatten(1)
    if fmt == "e4m3":
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
        c = torch.bucketize(q.abs(), edges).to(torch.uint8) + 8 * torch.signbit(q).to(torch.uint8)
        codes = c[:, 0::2] | (c[:, 1::2] << 4)
    pad = torch.nn.functional.pad
    scales = (e[:, :, 0] + 127).to(torch.uint8)
    return (pad(codes, (0, _code_bytes(k, fmt) - codes.shape[1])).contiguous(),
            pad(scales, (0, _scale_bytes(k) - scales.shape[1])).contiguous())


def _hidden(g, rows, k, dtype, size=1.0):
    """Hidden states: normal, with a few channels far larger than the others."""
    ch = torch.exp(0.5 * torch.randn(k, generator=g, device=DEV))
    ch[torch.randint(0, k, (max(1, k // 512),), generator=g, device=DEV)] *= 20
    return (torch.randn(rows, k, generator=g, device=DEV) * (ch * size)).to(dtype)


def _weight(g, d, k):
    """A weight in 4 bits, its output features of different sizes, products of order one."""
    w = torch.randn(d, k, generator=g, device=DEV) * torch.exp(0.3 * torch.randn(d, 1, generator=g, device=DEV))
    return _held(w * (0.7 * k ** -0.5), "e2m1")


def _logits(g, rows, experts):
    """A router's logits: some experts are favoured, and the batch's rows agree on it."""
    return 1.5 * torch.randn(rows, experts, generator=g, device=DEV) + torch.randn(experts, generator=g, device=DEV)


def _routing(g, rows, experts, top_k):
    """(ids [rows, top_k], weights): what a router hands on; a few rows of the batch are padding."""
    logits = _logits(g, rows, experts)
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    ids = ids[:, :top_k].int()
    ids[torch.rand(rows, generator=g, device=DEV) < 0.02] = -1
    return ids.contiguous(), torch.softmax(top[:, :top_k], 1).contiguous()


class _Weight:
    """A weight as the library keeps it, freed with the state that holds it."""

    def __init__(self, d, k, codes, scales):
        from rank_adapter_gemm_lora_amd import binding as lb
        self.lb = lb
        self.at = lb.lora_mx_weight_create(d, k)
        lb.lora_mx_weight_load_packed(self.at, codes.data_ptr(), codes.shape[1], scales.data_ptr(), scales.shape[1], _stream())

    def __del__(self):
        self.lb.lora_mx_weight_destroy(self.at)


class _Experts:
    """The experts' weights as the library keeps them."""

    def __init__(self, held, d, k, gated):
        from rank_adapter_gemm_lora_amd import binding as lb
        self.lb = lb
        self.at = lb.lora_mx_experts_create(len(held), d, k, gated)
        for e, (codes, scales) in enumerate(held):
            lb.lora_mx_experts_load_packed(self.at, e, codes.data_ptr(), codes.shape[1], scales.data_ptr(), scales.shape[1], _stream())

    def __del__(self):
        self.lb.lora_mx_experts_destroy(self.at)


class _Plan:
    """A batch's grouping by expert."""

    def __init__(self, rows, experts, top_k, ids=None):
        from rank_adapter_gemm_lora_amd import binding as lb
        self.lb = lb
        self.at = lb.lora_moe_plan_create(rows, experts, top_k)
        if ids is not None:
            lb.lora_moe_group(self.at, ids.data_ptr(), rows, 0, 0, _stream())

    def __del__(self):
        self.lb.lora_moe_plan_destroy(self.at)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _gated(c):
    return c.get("act") == "swiglu"


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c, rows, dt = case, case["rows"], DT[case["dtype"]]
    s = {"case": case}

    def empty(*shape, dtype=dt):
        return torch.zeros(*shape, dtype=dtype, device=DEV)

    def held(n, k, fmt="e4m3"):
        return empty(n, _code_bytes(k, fmt), dtype=torch.uint8), empty(n, _scale_bytes(k), dtype=torch.uint8)
    if c["op"] == "norm":
        k = c["k"]
        s["y"], s["r"] = _hidden(g, rows, k, dt), _hidden(g, rows, k, dt, 3.0)
        s["post"] = (0.5 + 0.2 * torch.randn(k, generator=g, device=DEV)).to(dt) if c["post"] else None
        s["pre"] = (1 + 0.2 * torch.randn(k, generator=g, device=DEV)).to(dt)
        s["gate"] = None if c["gate"] == "none" else torch.sigmoid(torch.randn(
            1 if c["gate"] == "channel" else rows, k, generator=g, device=DEV)).to(dt)
        s["scale"] = 0.75
        s["q"], s["s"] = held(rows, k)
        s["h"], s["out"], s["v"] = empty(rows, k), empty(rows, k), empty(rows, k)
        return s
    if c["op"] == "route":
        x, top_k = _logits(g, rows, c["experts"]), c["top_k"]
        if c["masked"]:   # experts that are switched off, and rows of padding
            x[:, torch.rand(c["experts"], generator=g, device=DEV) < 0.05] = -math.inf
            x[torch.rand(rows, generator=g, device=DEV) < 0.05] = -math.inf
        s["x"] = x.to(dt)
        s["ids"] = empty(rows, top_k, dtype=torch.int32)
        s["w"] = empty(rows, top_k, dtype=torch.float32)
        s["order"] = empty(rows * top_k, dtype=torch.int32)
        s["offsets"] = empty(c["experts"] + 1, dtype=torch.int32)
        if own:
            s["plan"] = _Plan(rows, c["experts"], top_k)
        return s
    if c["op"] == "fused":
        k, d = c["k"], c["d"]
        s["q"], s["s"] = _held(_hidden(g, rows, k, torch.float32), c["fmt"])
        s["wq"], s["ws"] = _weight(g, d, k)
        s["bias"] = torch.randn(d, generator=g, device=DEV).to(dt) if c["bias"] else None
        s["r"] = _hidden(g, rows, d, dt, 2.0) if c["residual"] else None
        s["y"] = empty(rows, d)
        if c["held"]:
            s["yq"], s["ys"] = held(rows, d)
        if own:
            s["w"] = _Weight(d, k, s["wq"], s["ws"])
        return s
    experts, top_k, f = c["experts"], c["top_k"], c["f"]
    s["ids"], s["w"] = _routing(g, rows, experts, top_k)
    s["counts"] = torch.bincount(s["ids"].flatten().long() + 1, minlength=experts + 1).tolist()
    if c["op"] == "up":
        d, k = (2 * f if _gated(c) else f), c["k"]
        x = _hidden(g, rows, k, torch.float32)
    else:
        d, k = c["d"], f
        x = torch.randn(rows * top_k, k, generator=g, device=DEV) * torch.exp(torch.randn(rows * top_k, k, generator=g, device=DEV))
    s["q"], s["s"] = _held(x, c["fmt"])
    s["held"] = [_weight(g, d, k) for _ in range(experts)]
    s["bias"] = torch.randn(experts, d, generator=g, device=DEV).to(dt) if c.get("bias") else None
    if c["op"] == "up":
        s["y"] = empty(rows * top_k, f)
        if c["held"]:
            s["yq"], s["ys"] = held(rows * top_k, f)
    else:
        s["y"], s["out"] = empty(rows * top_k, d), empty(rows, d)
        s["r"] = _hidden(g, rows, d, dt, 2.0) if c["residual"] else None
    if own:
        s["experts"] = _Experts(s["held"], d, k, _gated(c))
        s["plan"] = _Plan(rows, experts, top_k, s["ids"])
    return s


# ------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _grouped(ids, experts):
    """Pairs grouped by expert, in their own order inside a group; those without an expert last."""
    key = torch.where(ids < 0, experts, ids).flatten()
    return torch.sort(key, stable=True)[1]


def _run_plain(s):
    c = s["case"]
    dt = DT[c["dtype"]]
    if c["op"] == "norm":
        y = s["y"].float()
        if s["post"] is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["post"].float()
        h = s["r"].float() + s["scale"] * (y if s["gate"] is None else s["gate"].float() * y)
        n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["pre"].float()
        return {"h": h.to(dt), "out": n.to(dt), "held": _values(n).to(dt)}
    if c["op"] == "route":
        x, experts, top_k = s["x"].float(), c["experts"], c["top_k"]
        top, ids = torch.sort(x, dim=1, descending=True, stable=True)
        top, ids = top[:, :top_k], ids[:, :top_k].int()
        off = top == -math.inf
        ids = torch.where(off, -1, ids)
        if c["score"] == "softmax":
            w = torch.exp(top - torch.where(off[:, :1], 0.0, top[:, :1]))
        else:
            w = 1 / (1 + torch.exp(-top))
        w = torch.where(off, 0.0, w / torch.where(off[:, :1], 1.0, w.sum(1, keepdim=True)))
        counts = torch.bincount(ids.flatten().long() + 1, minlength=experts + 1)
        offsets = torch.cat((counts[:1] * 0, torch.cumsum(counts[1:], 0)))
        return {"ids": ids, "weights": w, "order": _grouped(ids, experts).int(), "offsets": offsets.int()}
    if c["op"] == "fused":
        y = _decode(s["q"], s["s"], c["fmt"], c["k"]) @ _decode(s["wq"], s["ws"], "e2m1", c["k"]).T
        if s["bias"] is not None:
            y = y + s["bias"].float()
        y = _act(y, c["act"])
        if s["r"] is not None:
            y = y + s["r"].float()
        return (_values(y) if c["held"] else y).to(dt)
    rows, top_k = c["rows"], c["top_k"]
    pairs = _grouped(s["ids"], c["experts"])
    k = c["k"] if c["op"] == "up" else c["f"]
    x = _decode(s["q"], s["s"], c["fmt"], k)
    parts, at = [], 0
    for e, n in enumerate(s["counts"][1:]):
        if n:
            a = x[pairs[at:at + n] // top_k] if c["op"] == "up" else x[at:at + n]
            y = a @ _decode(*s["held"][e], "e2m1", k).T
            if s["bias"] is not None:
                y = y + s["bias"][e].float()
            parts.append(_act(y, c.get("act")))
            at += n
    left = rows * top_k - at
    width = c["f"] if c["op"] == "up" else c["d"]
    if left:
        parts.append(torch.zeros(left, width, device=DEV))
    y = torch.cat(parts)
    if c["op"] == "up":
        return (_values(y) if c["held"] else y).to(dt)
    back = torch.empty_like(pairs)
    back[pairs] = torch.arange(len(pairs), device=DEV)
    w = torch.where(s["ids"] < 0, 0.0, s["w"])
    out = torch.zeros(rows, width, device=DEV) if s["r"] is None else s["r"].float()
    for j in range(top_k):
        out = out + w[:, j:j + 1] * y[back.view(rows, top_k)[:, j]]
    return out.to(dt)


def _run_own(s):
    from rank_adapter_gemm_lora_amd import binding as lb
    c, st = s["case"], _stream()
    rows = c["rows"]
    dt = lb.LORA_BF16 if c["dtype"] == "bf16" else lb.LORA_F32
    fmt = lb.LORA_MX_E2M1 if c.get("fmt") == "e2m1" else lb.LORA_MX_E4M3

    def at(t):
        return 0 if t is None else t.data_ptr()
    if c["op"] == "norm":
        k, held = c["k"], (s["q"].data_ptr(), s["q"].stride(0), s["s"].data_ptr(), s["s"].stride(0))
        lb.lora_block_norm_mx(s["out"].data_ptr(), k, *held, s["h"].data_ptr(), k, s["y"].data_ptr(), k, s["r"].data_ptr(), k,
                              at(s["post"]), at(s["gate"]), k if c["gate"] == "row" else 0, s["scale"], at(s["pre"]), EPS, dt,
                              rows, k, st)
        lb.lora_mx_dequantize(s["v"].data_ptr(), k, dt, *held, lb.LORA_MX_E4M3, rows, k, st)
        return {"h": s["h"], "out": s["out"], "held": s["v"]}
    if c["op"] == "route":
        lb.lora_moe_route(s["plan"].at, s["ids"].data_ptr(), s["w"].data_ptr(), s["order"].data_ptr(), s["offsets"].data_ptr(),
                          s["x"].data_ptr(), s["x"].stride(0), dt, rows,
                          lb.LORA_MOE_SOFTMAX if c["score"] == "softmax" else lb.LORA_MOE_SIGMOID, True, 1.0, st)
        return {"ids": s["ids"], "weights": s["w"], "order": s["order"], "offsets": s["offsets"]}
    x = (s["q"].data_ptr(), s["q"].stride(0), s["s"].data_ptr(), s["s"].stride(0), fmt)
    if c.get("held"):
        y = (0, 0, s["yq"].data_ptr(), s["yq"].stride(0), s["ys"].data_ptr(), s["ys"].stride(0))
    else:
        y = (s["y"].data_ptr(), s["y"].stride(0), 0, 0, 0, 0)
    act = {"none": lb.LORA_ACT_NONE, "relu": lb.LORA_ACT_RELU, "silu": lb.LORA_ACT_SILU, "gelu": lb.LORA_ACT_GELU,
           "gelu_tanh": lb.LORA_ACT_GELU_TANH, "swiglu": lb.LORA_ACT_SWIGLU}[c.get("act", "none")]
    if c["op"] == "fused":
        lb.lora_mx_linear_fused(s["w"].at, *y, dt, *x, at(s["bias"]), act, at(s["r"]), c["d"], rows, st)
    else:
        lb.lora_mx_expert_linear(s["experts"].at, s["plan"].at, *y, dt, *x,
                                 lb.LORA_MOE_ROWS if c["op"] == "up" else lb.LORA_MOE_PAIRS, at(s["bias"]), act, st)
    if c["op"] == "down":
        lb.lora_moe_combine(s["plan"].at, s["out"].data_ptr(), c["d"], s["y"].data_ptr(), c["d"], s["w"].data_ptr(), at(s["r"]),
                            c["d"], dt, c["d"], st)
        return s["out"]
    if c["held"]:
        lb.lora_mx_dequantize(s["y"].data_ptr(), s["y"].stride(0), dt, *y[2:], lb.LORA_MX_E4M3, len(s["y"]), s["y"].shape[1], st)
    return s["y"]


# ------------------------------------------------------------- in 64 bits

def _nearest(v):
    """The values that [rows, k] stands for in e4m3 blocks, by search among the format's values."""
    rows, k = v.shape
    n = -(-k // 32)
    b = torch.zeros(rows, n * 32, dtype=torch.float64, device=v.device)
    b[:, :k] = v
    b = b.view(rows, n, 32)
    peak = b.abs().max(-1, keepdim=True).values
    # the binade of the largest: log2 may round up onto a power of two
    lg = torch.floor(torch.log2(peak.clamp(min=2.0 ** -140)))
    lg = lg - (torch.exp2(lg) > peak).double() + (torch.exp2(lg + 1) <= peak).double()
    scale = torch.exp2((lg - 8).clamp(-127, 127))
    grid = torch.arange(127, dtype=torch.uint8, device=v.device).view(torch.float8_e4m3fn).double()
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


def _act64(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v * torch.special.expit(v)
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "gelu_tanh":   # (1 + tanh z) / 2 is the logistic function of 2 z
        return v * torch.special.expit(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if act == "swiglu":
        f = v.shape[1] // 2
        return v[:, :f] * torch.special.expit(v[:, :f]) * v[:, f:]
    return v


def _rms(v):
    return v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / v.shape[1] + EPS)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        a = s["y"].double()
        if c["post"]:
            a = _rms(a) * s["post"].double()
        if s["gate"] is not None:
            a = a * s["gate"].double()
        h = a * s["scale"] + s["r"].double()
        n = _rms(h) * s["pre"].double()
        return {"h": h, "out": n, "held": _nearest(n)}
    if c["op"] == "route":
        x, experts = s["x"].double(), c["experts"]
        left, number, chosen, score = x.clone(), torch.arange(experts, device=DEV), [], []
        for _ in range(c["top_k"]):   # the largest that is left, the lowest number among equals
            top = left.max(1, keepdim=True).values
            i = torch.where(left == top, number, experts).min(1, keepdim=True).values
            none = top == -math.inf
            p = torch.exp(top - x.max(1, keepdim=True).values) if c["score"] == "softmax" else torch.special.expit(top)
            score.append(torch.where(none, 0.0, p))
            chosen.append(torch.where(none, -1, i))
            left.scatter_(1, i, -math.inf)
        ids, p = torch.cat(chosen, 1), torch.cat(score, 1)
        total = p.sum(1, keepdim=True)
        flat = ids.flatten()
        order = torch.cat([(flat == e).nonzero()[:, 0] for e in list(range(experts)) + [-1]])
        offsets = torch.stack([((flat >= 0) & (flat < e)).sum() for e in range(experts + 1)])
        return {"ids": ids.int(), "weights": torch.where(total > 0, p / total, 0.0), "order": order.int(),
                "offsets": offsets.int()}
    if c["op"] == "fused":
        y = torch.matmul(_meant(s["q"], s["s"], c["fmt"], c["k"]), _meant(s["wq"], s["ws"], "e2m1", c["k"]).t())
        y = _act64(y if s["bias"] is None else y + s["bias"].double(), c["act"])
        y = y if s["r"] is None else y + s["r"].double()
        return _nearest(y) if c["held"] else y
    rows, top_k, flat = c["rows"], c["top_k"], s["ids"].flatten()
    k, width = (c["k"], c["f"]) if c["op"] == "up" else (c["f"], c["d"])
    x = _meant(s["q"], s["s"], c["fmt"], k)
    y = torch.zeros(rows * top_k, width, dtype=torch.float64, device=DEV)
    out = torch.zeros(rows, width, dtype=torch.float64, device=DEV)
    at = 0
    for e in range(c["experts"]):
        mine = (flat == e).nonzero()[:, 0]
        n, row = len(mine), mine // top_k
        v = torch.matmul(x[row] if c["op"] == "up" else x[at:at + n], _meant(*s["held"][e], "e2m1", k).t())
        v = _act64(v if s["bias"] is None else v + s["bias"][e].double(), c.get("act"))
        y[at:at + n] = v
        if c["op"] == "down":
            out.index_add_(0, row, v * s["w"].flatten()[mine, None].double())
        at += n
    if c["op"] == "down":
        return out if s["r"] is None else out + s["r"].double()
    return _nearest(y) if c["held"] else y


# ------------------------------------------------------------- what a pass needs

def work(case):
    c = case
    rows, e = c["rows"], 2 if c["dtype"] == "bf16" else 4
    per, w = {"e4m3": 1.0, "e2m1": 0.5}.get(c.get("fmt"), 0.0) + 1 / 32, 0.5 + 1 / 32   # bytes an element held in blocks takes
    if c["op"] == "norm":
        k = c["k"]
        gate = {"none": 0, "channel": k, "row": rows * k}[c["gate"]]
        return {"bytes": e * (5 * rows * k + gate + (2 if c["post"] else 1) * k), "flops": 16 * rows * k}
    if c["op"] == "route":
        return {"bytes": rows * (c["experts"] * e + c["top_k"] * 12) + 4 * c["experts"] + 4,
                "flops": rows * c["experts"] * c["top_k"]}
    if c["op"] == "fused":
        k, d = c["k"], c["d"]
        return {"bytes": rows * k * per + d * k * w + rows * d * e * (2 if c["residual"] else 1) + (d * e if c["bias"] else 0),
                "flops": 2 * rows * k * d}
    pairs, f = rows * c["top_k"], c["f"]
    used = min(c["experts"], pairs)
    if c["op"] == "up":
        k, d = c["k"], (2 * f if _gated(c) else f)
        return {"bytes": rows * k * per + used * (d * k * w + (d * e if c["bias"] else 0)) + pairs * (f * e + 4),
                "flops": 2 * pairs * k * d}
    d = c["d"]
    return {"bytes": pairs * (f * per + 8) + used * d * f * w + rows * d * e * (2 if c["residual"] else 1),
            "flops": 2 * pairs * f * d}
