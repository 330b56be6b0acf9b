"""One decoder layer with a mixture MLP: 4-bit base weights and experts, LoRA adapters on q/k/v.

    python examples/mixture_layer.py [--rows 64] [--experts 64] [--top-k 8]

    qkv = Wqkv x + bias                          lora_mx_linear_fused
    qkv += the rows' adapters on x               lora_build_apply
    (attention: the caller's; here its output is a tensor that is passed in)
    o = Wo attention                             lora_mx_quantize, lora_mx_linear_fused
    residual += norm(o);  x = norm(residual)     lora_block_norm_mx: x in bf16 and in 8-bit blocks
    logits = R x                                 (a plain product of the caller's)
    experts, weights, groups                     lora_moe_route
    a = silu(gate) * up, in blocks               lora_mx_expert_linear
    y = the experts' second products             lora_mx_expert_linear
    m = sum of weight * y                        lora_moe_combine
    residual += norm(m);  x = norm(residual)     lora_block_norm_mx: the next layer's input

All buffers are made once; step() only launches, so it can be captured in a
HIP graph.
"""
import argparse
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [p for p in (HERE, os.path.dirname(HERE)) if p not in sys.path]

import torch

from mx_layer import BF, E4M3, Blocks, Projection, _stream
from rank_adapter_gemm_lora_amd import binding as lb

F32 = lb.LORA_F32


class Experts:
    """Weights of all experts: [experts][d][k] bf16 on the GPU."""

    def __init__(self, weights, gated):
        n, d, k = weights.shape
        self.at = lb.lora_mx_experts_create(n, d, k, gated)
        for e in range(n):
            lb.lora_mx_experts_load(self.at, e, weights[e].data_ptr(), weights.stride(1), BF, _stream())

    def close(self):
        lb.lora_mx_experts_destroy(self.at)


class MixtureLayer:
    def __init__(self, w, max_rows, top_k, n_slots, r_max, eps=1e-5):
        """w, bf16 on the GPU: "qkv" [dq + 2 dkv][k], "bias" [dq + 2 dkv], "o" [k][dq], "router" [experts][k], "up" [experts][2
        f][k] (gates first), "down" [experts][k][f], and the norms "post_attention", "pre_mlp", "post_mlp", "next" [k]; the
        q/k/v widths are w["slices"]."""
        dev = w["qkv"].device
        self.w, self.eps, self.top_k = w, eps, top_k
        self.k, self.dq, self.experts, self.f = w["qkv"].shape[1], w["o"].shape[1], w["down"].shape[0], w["down"].shape[2]
        self.qkv = Projection(w["qkv"], max_rows, w["slices"], n_slots, r_max)
        self.o = Projection(w["o"], max_rows)
        self.up, self.down = Experts(w["up"], True), Experts(w["down"], False)
        self.plan = lb.lora_moe_plan_create(max_rows, self.experts, top_k)
        pairs = max_rows * top_k

        def buf(n, width, dtype=torch.bfloat16):
            return torch.zeros(n, width, dtype=dtype, device=dev)
        self.y_qkv, self.y_o, self.x, self.m = (buf(max_rows, d) for d in (self.qkv.d, self.k, self.k, self.k))
        self.bo, self.bx, self.ba = Blocks(max_rows, self.dq, dev), Blocks(max_rows, self.k, dev), Blocks(pairs, self.f, dev)
        self.y = buf(pairs, self.k, torch.float32)
        self.logits, self.ids = buf(max_rows, self.experts), buf(max_rows, top_k, torch.int32)
        self.weights = buf(max_rows, top_k, torch.float32)

    def _norm(self, x, blocks, y, residual, post, pre, rows):
        k = self.k
        lb.lora_block_norm_mx(x.data_ptr(), k, *blocks.args, residual.data_ptr(), k, y.data_ptr(), k, residual.data_ptr(), k,
                              self.w[post].data_ptr(), 0, 0, 1.0, self.w[pre].data_ptr(), self.eps, BF, rows, k, _stream())

    def _fused(self, p, y, blocks, bias, rows):
        lb.lora_mx_linear_fused(p.w, y.data_ptr(), y.stride(0), 0, 0, 0, 0, BF, *blocks.args, E4M3,
                                0 if bias is None else bias.data_ptr(), lb.LORA_ACT_NONE, 0, 0, rows, _stream())

    def begin(self, x, blocks, ids, rows):
        """q, k and v of the batch (self.y_qkv) from the normed input in both forms; ids: the rows' adapters."""
        st, p = _stream(), self.qkv
        self._fused(p, self.y_qkv, blocks, self.w["bias"], rows)
        lb.lora_build_apply(p.stack, self.y_qkv.data_ptr(), p.d, x.data_ptr(), x.stride(0), ids.data_ptr(), rows, p.seg, st)

    def finish(self, attention, x, blocks, residual, rows):
        """From attention's output to the next layer's normed input (into x and blocks); residual moves on."""
        st, k, w = _stream(), self.k, self.w
        lb.lora_mx_quantize(*self.bo.args, E4M3, attention.data_ptr(), attention.stride(0), BF, rows, self.dq, st)
        self._fused(self.o, self.y_o, self.bo, None, rows)
        self._norm(self.x, self.bx, self.y_o, residual, "post_attention", "pre_mlp", rows)
        torch.mm(self.x[:rows], w["router"].t(), out=self.logits[:rows])
        lb.lora_moe_route(self.plan, self.ids.data_ptr(), self.weights.data_ptr(), 0, 0, self.logits.data_ptr(), self.experts, BF,
                          rows, lb.LORA_MOE_SOFTMAX, True, 1.0, st)
        lb.lora_mx_expert_linear(self.up.at, self.plan, 0, 0, *self.ba.args, BF, *self.bx.args, E4M3, lb.LORA_MOE_ROWS, 0,
                                 lb.LORA_ACT_SWIGLU, st)
        lb.lora_mx_expert_linear(self.down.at, self.plan, self.y.data_ptr(), k, 0, 0, 0, 0, F32, *self.ba.args, E4M3,
                                 lb.LORA_MOE_PAIRS, 0, lb.LORA_ACT_NONE, st)
        lb.lora_moe_combine(self.plan, self.m.data_ptr(), k, self.y.data_ptr(), k, F32, self.weights.data_ptr(), 0, 0, BF, k, st)
        self._norm(x, blocks, self.m, residual, "post_mlp", "next", rows)

    def step(self, x, blocks, residual, ids, rows):
        """Both halves with q standing in for attention's output."""
        self.begin(x, blocks, ids, rows)
        self.finish(self.y_qkv[:, :self.dq], x, blocks, residual, rows)

    def close(self):
        lb.lora_moe_plan_destroy(self.plan)
        for p in (self.qkv, self.o, self.up, self.down):
            p.close()


def random_layer(k, slices, f, experts, top_k, max_rows, n_slots, rank, seed=0, device="cuda:0"):
    """A layer of random weights with an adapter in every slot."""
    g = torch.Generator(device=device).manual_seed(seed)

    def rand(*shape, std):
        return (torch.randn(*shape, generator=g, device=device) * std).bfloat16()
    dq, d = slices[0], sum(slices)
    w = {"qkv": rand(d, k, std=k ** -0.5), "bias": rand(d, std=0.5), "o": rand(k, dq, std=dq ** -0.5),
         "router": rand(experts, k, std=2 * k ** -0.5), "up": rand(experts, 2 * f, k, std=k ** -0.5),
         "down": rand(experts, k, f, std=f ** -0.5), "slices": slices}
    w.update({n: 1 + rand(k, std=0.1) for n in ("post_attention", "pre_mlp", "post_mlp", "next")})
    layer = MixtureLayer(w, max_rows, top_k, n_slots, rank)
    adapters = {}
    for s in range(n_slots):
        A, B = rand(len(slices), rank, k, std=k ** -0.5), rand(d, rank, std=0.1)
        layer.qkv.load(s, A, B, 2.0 * rank)
        adapters["qkv", s] = (A, B, 2.0)   # scale alpha / rank
    torch.cuda.synchronize()
    return layer, w, adapters


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=64)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--adapters", type=int, default=8)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args()
    k, slices, f, dev = 4096, [4096, 1024, 1024], 1024, "cuda:0"
    layer, _, _ = random_layer(k, slices, f, a.experts, a.top_k, a.rows, a.adapters, a.rank)
    g = torch.Generator(device=dev).manual_seed(1)
    x, residual = (torch.randn(a.rows, k, generator=g, device=dev).bfloat16() for _ in range(2))
    ids = torch.randint(-1, a.adapters, (a.rows,), generator=g, device=dev, dtype=torch.int32)
    blocks = Blocks(a.rows, k, dev)
    lb.lora_mx_quantize(*blocks.args, E4M3, x.data_ptr(), k, BF, a.rows, k, _stream())
    for _ in range(3):
        layer.step(x, blocks, residual, ids, a.rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(x, blocks, residual, ids, a.rows)
    for run, name in ((lambda: layer.step(x, blocks, residual, ids, a.rows), "launched"), (graph.replay, "graph replay")):
        run()
        torch.cuda.synchronize()
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        for _ in range(a.steps):
            run()
        t1.record()
        torch.cuda.synchronize()
        print(f"{a.rows} rows, top {a.top_k} of {a.experts} experts: {t0.elapsed_time(t1) / a.steps * 1e3:.1f} us a layer ({name})")
    layer.close()


if __name__ == "__main__":
    main()
