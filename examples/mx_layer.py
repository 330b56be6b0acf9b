"""One decoder layer's projections with 4-bit base weights and LoRA adapters.

    python examples/mx_layer.py [--rows 64] [--adapters 8] [--rank 16]

The base weights are held in 4 bits (e2m1 blocks) and shared by the batch; each
row's adapter adds its delta in bf16.  One pass over the hidden state gives both
forms that the two need:

    residual += hidden;  x = norm(residual)      lora_rmsnorm_mx: x in bf16 and in 8-bit blocks
    qkv = Wqkv x                                 lora_mx_linear on the blocks
    qkv += the rows' adapters on x               lora_build_apply on the bf16 form
    (attention: the caller's; here its output is a tensor that is passed in)
    o = Wo attention                             lora_mx_quantize, lora_mx_linear
    residual += o;  x = norm(residual)           lora_rmsnorm_mx
    gu = Wgu x, += adapters                      lora_mx_linear, lora_build_apply
    a = silu(gate) * up                          lora_swiglu_mx: bf16 and blocks
    hidden = Wdown a, += adapters                lora_mx_linear, lora_build_apply

All buffers are made once; step() only launches, so it can be captured in a
HIP graph.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

from rank_adapter_gemm_lora_amd import binding as lb

BF, E4M3 = lb.LORA_BF16, lb.LORA_MX_E4M3


def _stream():
    return torch.cuda.current_stream().cuda_stream


class Blocks:
    """Rows in 8-bit blocks."""

    def __init__(self, rows, k, device):
        self.q = torch.zeros(rows, lb.lora_mx_code_bytes(k, E4M3), dtype=torch.uint8, device=device)
        self.s = torch.zeros(rows, lb.lora_mx_scale_bytes(k), dtype=torch.uint8, device=device)
        self.args = (self.q.data_ptr(), self.q.stride(0), self.s.data_ptr(), self.s.stride(0))


class Projection:
    """A base weight in 4 bits and, where slices are given, a stack of adapters next to it."""

    def __init__(self, weight, max_rows, slices=None, n_slots=0, r_max=0):
        d, k = weight.shape
        self.d, self.k, self.n_slots = d, k, n_slots
        self.w = lb.lora_mx_weight_create(d, k)
        lb.lora_mx_weight_load(self.w, weight.data_ptr(), weight.stride(0), BF, _stream())
        self.stack = self.seg = None
        if slices:
            self.stack = lb.lora_stack_create(BF, n_slots, r_max, k, slices, max_rows)
            self.seg = lb.lora_segments_create(max_rows, n_slots)

    def load(self, slot, A, B, alpha):
        """Adapter: A [slices][rank][k], B [d][rank], bf16 on the GPU."""
        lb.lora_load_slot(self.stack, slot, A.shape[1], alpha, A.data_ptr(), B.data_ptr(), False, _stream())

    def run(self, y, x, blocks, ids, rows):
        st = _stream()
        lb.lora_mx_linear(self.w, y.data_ptr(), y.stride(0), BF, *blocks.args, E4M3, rows, st)
        if self.stack is not None:
            lb.lora_build_apply(self.stack, y.data_ptr(), y.stride(0), x.data_ptr(), x.stride(0), ids.data_ptr(), rows,
                                self.seg, st)

    def close(self):
        if self.stack is not None:
            lb.lora_segments_destroy(self.seg)
            lb.lora_stack_destroy(self.stack)
        lb.lora_mx_weight_destroy(self.w)


class MxLayer:
    def __init__(self, w, max_rows, n_slots, r_max, eps=1e-5):
        """w: {"qkv": [dq + 2 dkv][k], "o": [k][dq], "gu": [2 f][k], "down": [k][f], "norm1", "norm2": [k]}, bf16
        on the GPU; the q/k/v widths are w["slices"]."""
        dev = w["qkv"].device
        self.k, self.f, self.dq, self.eps = w["qkv"].shape[1], w["down"].shape[1], w["o"].shape[1], eps
        self.norm1, self.norm2 = w["norm1"], w["norm2"]
        self.qkv = Projection(w["qkv"], max_rows, w["slices"], n_slots, r_max)
        self.o = Projection(w["o"], max_rows)
        self.gu = Projection(w["gu"], max_rows, [self.f, self.f], n_slots, r_max)
        self.down = Projection(w["down"], max_rows, [self.k], n_slots, r_max)

        def buf(width):
            return torch.zeros(max_rows, width, dtype=torch.bfloat16, device=dev)
        self.x1, self.x2, self.a = buf(self.k), buf(self.k), buf(self.f)
        self.y_qkv, self.y_o, self.y_gu = buf(self.qkv.d), buf(self.k), buf(2 * self.f)
        self.b1, self.b2 = Blocks(max_rows, self.k, dev), Blocks(max_rows, self.k, dev)
        self.bo, self.ba = Blocks(max_rows, self.dq, dev), Blocks(max_rows, self.f, dev)

    def _norm(self, x, blocks, hidden, residual, weight, rows):
        k = self.k
        lb.lora_rmsnorm_mx(x.data_ptr(), k, *blocks.args, residual.data_ptr(), residual.stride(0), hidden.data_ptr(),
                           hidden.stride(0), residual.data_ptr(), residual.stride(0), weight.data_ptr(), self.eps, BF,
                           rows, k, _stream())

    def begin(self, hidden, residual, ids, rows):
        """q, k and v of the batch (self.y_qkv); residual becomes residual + hidden."""
        self._norm(self.x1, self.b1, hidden, residual, self.norm1, rows)
        self.qkv.run(self.y_qkv, self.x1, self.b1, ids, rows)

    def finish(self, attention, hidden, residual, ids, rows):
        """From attention's output to the layer's (into hidden); residual moves on too."""
        lb.lora_mx_quantize(*self.bo.args, E4M3, attention.data_ptr(), attention.stride(0), BF, rows, self.dq, _stream())
        self.o.run(self.y_o, None, self.bo, ids, rows)
        self._norm(self.x2, self.b2, self.y_o, residual, self.norm2, rows)
        self.gu.run(self.y_gu, self.x2, self.b2, ids, rows)
        lb.lora_swiglu_mx(self.a.data_ptr(), self.f, *self.ba.args, self.y_gu.data_ptr(), 2 * self.f, BF, rows, self.f,
                          _stream())
        self.down.run(hidden, self.a, self.ba, ids, rows)

    def step(self, hidden, residual, ids, rows):
        """Both halves with q standing in for attention's output."""
        self.begin(hidden, residual, ids, rows)
        self.finish(self.y_qkv[:, :self.dq], hidden, residual, ids, rows)

    def close(self):
        for p in (self.qkv, self.o, self.gu, self.down):
            p.close()


def random_layer(k, slices, f, max_rows, n_slots, rank, seed=0, device="cuda:0"):
    """A layer of random weights with an adapter in every slot."""
    g = torch.Generator(device=device).manual_seed(seed)

    def rand(*shape, std):
        return (torch.randn(*shape, generator=g, device=device) * std).bfloat16()
    dq = slices[0]
    w = {"qkv": rand(sum(slices), k, std=k ** -0.5), "o": rand(k, dq, std=dq ** -0.5), "gu": rand(2 * f, k, std=k ** -0.5),
         "down": rand(k, f, std=f ** -0.5), "norm1": 1 + rand(k, std=0.1), "norm2": 1 + rand(k, std=0.1), "slices": slices}
    layer = MxLayer(w, max_rows, n_slots, rank)
    adapters = {}
    for name, p, n in (("qkv", layer.qkv, len(slices)), ("gu", layer.gu, 2), ("down", layer.down, 1)):
        for s in range(n_slots):
            A, B = rand(n, rank, p.k, std=p.k ** -0.5), rand(p.d, rank, std=0.1)
            p.load(s, A, B, 2.0 * rank)
            adapters[name, s] = (A, B, 2.0)   # scale alpha / rank
    torch.cuda.synchronize()
    return layer, w, adapters


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rows", type=int, default=64)
    ap.add_argument("--adapters", type=int, default=8)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args()
    k, slices, f = 4096, [4096, 1024, 1024], 14336
    layer, _, _ = random_layer(k, slices, f, a.rows, a.adapters, a.rank)
    g = torch.Generator(device="cuda:0").manual_seed(1)
    hidden = torch.randn(a.rows, k, generator=g, device="cuda:0").bfloat16()
    residual = torch.randn(a.rows, k, generator=g, device="cuda:0").bfloat16()
    ids = torch.randint(-1, a.adapters, (a.rows,), generator=g, device="cuda:0", dtype=torch.int32)
    for _ in range(3):
        layer.step(hidden, residual, ids, a.rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(hidden, residual, ids, a.rows)
    for run, name in ((lambda: layer.step(hidden, residual, ids, a.rows), "launched"), (graph.replay, "graph replay")):
        run()
        torch.cuda.synchronize()
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        for _ in range(a.steps):
            run()
        t1.record()
        torch.cuda.synchronize()
        print(f"{a.rows} rows, {a.adapters} adapters of rank {a.rank}: {t0.elapsed_time(t1) / a.steps * 1e3:.1f} us a layer ({name})")
    layer.close()


if __name__ == "__main__":
    main()
