"""One decode step of a small mixture-of-experts transformer, every product on
quantized weights: RMS norm (8-bit output) -> q/k/v -> cache store -> attention
over the paged cache -> output projection -> RMS norm with the residual's
addition -> routing -> expert products -> weighted sum.

Run on a GPU:  python examples/moe_decode_step.py
It decodes a few tokens for a batch of sequences of different lengths, prints
the time of a step (captured in a HIP graph and replayed), and `main` returns
the last hidden states for a caller to check.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from dequant_quantized_gemv_amd import qk, synth  # noqa: E402


class Layer:
    """Synthetic weights of one layer; `width` hidden, `inner` per expert."""

    def __init__(self, width=512, q_heads=8, kv_heads=2, dim=64, experts=16, used=4, inner=256, groups=4, fmt="q4_0",
                 seed=1, device="cuda"):
        self.width, self.q_heads, self.kv_heads, self.dim = width, q_heads, kv_heads, dim
        self.experts, self.used, self.inner, self.groups, self.fmt = experts, used, inner, groups, fmt
        self.device = device
        scales = (2.0 ** -7, 2.0 ** -6)  # activations stay near 1
        self.tensors = 0

        def matrix(rows, k):
            self.tensors += 1
            return torch.from_numpy(synth.quant_matrix(fmt, rows, k, seed=seed, tensor_id=self.tensors,
                                                       d_range=scales)).to(device)

        self.wq, self.wk, self.wv = (matrix(h * dim, width) for h in (q_heads, kv_heads, kv_heads))
        self.wo = matrix(width, q_heads * dim)
        self.wr = matrix(experts, width)
        self.gate, self.up = matrix(experts * inner, width), matrix(experts * inner, width)
        self.down = matrix(experts * width, inner)
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        self.norm1, self.norm2 = (1 + 0.1 * torch.randn(width, generator=g) for _ in range(2))
        self.norm1, self.norm2 = self.norm1.to(device), self.norm2.to(device)
        self.bias = (0.05 * torch.randn(experts, generator=g)).to(device)

    def step(self, x, cache, table, lens, workspace, window=0, sinks=0, max_len=None):
        """Hidden states (n, width) of the new token of each of n <= 8
        sequences, stored at position lens - 1 of the cache; new hidden states."""
        n, fmt, dim = x.shape[0], self.fmt, self.dim
        h8 = qk.rms_norm(x, self.norm1, out_dtype="x8")  # quantized once, used by three products
        q = qk.mul_mat_vec_x8q(fmt, self.wq, self.q_heads * dim, self.width, h8)
        k = qk.mul_mat_vec_x8q(fmt, self.wk, self.kv_heads * dim, self.width, h8)
        v = qk.mul_mat_vec_x8q(fmt, self.wv, self.kv_heads * dim, self.width, h8)
        qk.kv_store(cache, k.view(n, self.kv_heads, dim), v.view(n, self.kv_heads, dim), table, lens - 1)
        a = qk.attn_decode(cache, q.view(n, self.q_heads, dim), table, lens, window=window, sinks=sinks,
                           max_len=max_len, workspace=workspace)
        o = qk.mul_mat_vec(fmt, self.wo, self.width, self.q_heads * dim, a.view(n, -1))
        h, x = qk.rms_norm(o, self.norm2, residual=x)
        logits = qk.mul_mat_vec(fmt, self.wr, self.experts, self.width, h)
        ids, w = qk.moe_route(logits, self.used, score="sigmoid", bias=self.bias, n_groups=self.groups,
                              topk_groups=self.groups // 2, group_top=2)
        gate = qk.mul_mat_vec_id(fmt, self.gate, self.experts, self.inner, self.width, ids, h)
        up = qk.mul_mat_vec_id(fmt, self.up, self.experts, self.inner, self.width, ids, h)
        y = qk.mul_mat_vec_id(fmt, self.down, self.experts, self.width, self.inner, ids,
                              torch.nn.functional.silu(gate) * up)
        return x + (y * w[..., None]).sum(1)


def main(steps=4, kind="i8", page=16, lens=(1, 9, 30, 200), seed=1, time_it=True, record=None):
    layer = Layer(seed=seed)
    n, most = len(lens), max(lens) + steps
    per = -(-most // page)
    cache = qk.KVCache.empty(n * per, layer.kv_heads, page, layer.dim, kind)
    g = torch.Generator(device="cpu")
    g.manual_seed(seed + 1)
    table = torch.randperm(n * per, generator=g).to(torch.int32).view(n, per).cuda()
    # what the sequences hold already
    seq = torch.cat([torch.full((c,), i) for i, c in enumerate(lens)]).to(torch.int32).cuda()
    pos = torch.cat([torch.arange(c) for c in lens]).to(torch.int32).cuda()
    past = [torch.randn(len(seq), layer.kv_heads, layer.dim, generator=g).cuda() for _ in range(2)]
    qk.kv_store(cache, past[0], past[1], table, pos, seq=seq)
    workspace = qk.attn_decode_workspace(cache, n, layer.q_heads, most)
    x = torch.randn(n, layer.width, generator=g).cuda()
    now = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for _ in range(steps):
        now = now + 1
        x_in, x = x, layer.step(x, cache, table, now, workspace, max_len=most)
        if record is not None:
            record.append((x_in, x, now))
    if time_it:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(graph, stream=s):
                layer.step(x, cache, table, now, workspace, max_len=most)
        torch.cuda.current_stream().wait_stream(s)
        graph.replay()
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        for _ in range(20):
            graph.replay()
        e[1].record()
        torch.cuda.synchronize()
        print(f"one layer's decode step, {n} sequences: {e[0].elapsed_time(e[1]) / 20 * 1e3:.1f} us", flush=True)
    return x, layer, (past, seq, pos)


if __name__ == "__main__":
    out, *_ = main()
    print("hidden states", tuple(out.shape), "rms", float(out.square().mean().sqrt()))
