"""One decoder layer served from a paged 8-bit cache: prompts, then single tokens replayed from a CUDA graph.

    python examples/decoder_layer.py [--steps N]

Layer: RMSNorm -> fused Q4_K projection to queries, keys and values -> per-head norm and rotation ->
append to the cache -> attention over it -> Q4_K output projection with the residual -> RMSNorm ->
router and MoE block. Weights are random, in the sizes below.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_moe_q4k_gb300 as q4k  # noqa: E402

EPS = 1e-6


class Cache:
    """Pages for a fixed set of sequences: sequence i owns the pages of row i of the table."""

    def __init__(self, batch, max_len, kv_heads, head_dim, page=64):
        self.page, self.max_pages = page, -(-max_len // page)
        self.pages = batch * self.max_pages
        shape = (self.pages, kv_heads, page, head_dim)
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
        self.k_scale, self.v_scale = (torch.ones(shape[:2], device="cuda") for _ in range(2))
        self.table = torch.arange(self.pages, dtype=torch.int32, device="cuda").view(batch, self.max_pages)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")  # cached tokens, the call's new ones included


class DecoderLayer:
    def __init__(self, hidden=1024, q_heads=8, kv_heads=2, head_dim=128, experts=16, top_k=4, inter=512, seed=0):
        self.hidden, self.hq, self.hk, self.d = hidden, q_heads, kv_heads, head_dim
        self.experts, self.top_k, self.inter = experts, top_k, inter
        g = torch.Generator("cuda").manual_seed(seed)

        def slab(count, n, k):  # [count][n][k/256] Q4_K blocks
            out = torch.empty(count * n * (k // 256) * 144, dtype=torch.uint8, device="cuda")
            q4k.q4k_quantize_rows(torch.randn((count * n, k), device="cuda", generator=g) * k ** -0.5, count * n, k, out)
            return out

        def gain(n):
            return (1 + 0.1 * torch.randn(n, device="cuda", generator=g)).bfloat16().view(torch.int16)
        self.row = (q_heads + 2 * kv_heads) * head_dim
        self.w_qkv, self.w_o = slab(1, self.row, hidden), slab(1, hidden, q_heads * head_dim)
        self.w_gate, self.w_up, self.w_down = slab(experts, inter, hidden), slab(experts, inter, hidden), slab(experts, hidden, inter)
        self.w_router = torch.randn((experts, hidden), device="cuda", generator=g).bfloat16().view(torch.int16)
        self.n_in, self.n_post, self.n_q, self.n_k = gain(hidden), gain(hidden), gain(head_dim), gain(head_dim)
        self.inv_freq = 1e6 ** (-torch.arange(head_dim // 2, dtype=torch.float64, device="cuda") * 2 / head_dim)
        self.flag = torch.zeros(1, dtype=torch.int32, device="cuda")

    def buffers(self, m, batch):
        """What one call of `forward` writes; kept by the caller, so that a captured graph can be replayed."""
        def f(*shape):
            return torch.empty(shape, device="cuda")

        def ws(nbytes):
            return torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
        n, qw = self.hidden, self.hq * self.d
        return {"h": f(m, n), "qkv": f(m, self.row), "q": f(m, qw), "att": f(m, qw), "o": f(m, n), "mid": f(m, n), "y": f(m, n),
                "zero": torch.zeros(m, dtype=torch.int32, device="cuda"), "one": torch.ones(m, device="cuda"),
                "gemv": ws(max(q4k.q4k_moe_workspace_size(m, 1, 1, self.row, n), q4k.q4k_moe_workspace_size(m, 1, 1, n, qw))),
                "attn": ws(q4k.q4k_paged_attention_workspace_size(batch, m, self.hq, self.hk, self.d)),
                "moe": ws(q4k.q4k_moe_layer_routed_workspace_size(m, self.top_k, self.experts, n, self.inter, 0))}

    def forward(self, x, pos, q_start, cache, max_q_len, max_len, b):
        """x [m, hidden]: the new tokens of all sequences, q_start [batch + 1] their first rows, pos [m] their positions
        in their sequences; cache.lens already counts them. Returns the layer's output [m, hidden], in b["y"]."""
        m, n, hq, hk, d, row, qw = x.shape[0], self.hidden, self.hq, self.hk, self.d, self.row, self.hq * self.d
        where = (q_start, cache.lens, cache.table, cache.lens.numel(), cache.max_pages, cache.page, cache.pages)
        q4k.q4k_rms_norm(x, self.n_in, m, n, EPS, b["h"])
        q4k.q4k_moe_id_gemv(self.w_qkv, 0, 1, b["h"], n, 0, b["zero"], m, 1, row, n, b["qkv"], b["gemv"], b["gemv"].numel(), self.flag)
        keys, values = b["qkv"][:, qw:], b["qkv"][:, qw + hk * d:]
        q4k.q4k_qk_norm_rope(b["qkv"], None, m, hq, 0, d, row, row, self.n_q, None, EPS, pos, self.inv_freq, d, q4k.ROPE_HALVES,
                             b["q"], None, qw, qw)
        q4k.q4k_kv_append(keys, values, m, hk, d, row, row, self.n_k, EPS, self.inv_freq, d, q4k.ROPE_HALVES, *where,
                          cache.k, cache.v, cache.k_scale, cache.v_scale, self.flag)
        q4k.q4k_paged_attention(b["q"], m, hq, hk, d, qw, cache.k, cache.v, cache.k_scale, cache.v_scale, *where, max_q_len,
                                max_len, d ** -0.5, 0, b["att"], qw, b["attn"], b["attn"].numel(), self.flag)
        q4k.q4k_moe_id_gemv(self.w_o, 0, 1, b["att"], qw, 0, b["zero"], m, 1, n, qw, b["o"], b["gemv"], b["gemv"].numel(), self.flag)
        q4k.moe_combine_residual(x, b["o"], b["one"], None, None, q4k.SHARED_NONE, m, 1, n, b["mid"])
        q4k.q4k_rms_norm(b["mid"], self.n_post, m, n, EPS, b["h"])
        q4k.q4k_moe_layer_forward_routed(self.w_gate, self.w_up, self.w_down, self.experts, None, None, None, 0, q4k.SHARED_NONE,
                                         b["h"], b["mid"], self.w_router, None, None, q4k.ROUTE_SOFTMAX, True, 1.0, 1, 1, m,
                                         self.top_k, n, self.inter, b["y"], None, EPS, None, None, None, b["moe"],
                                         b["moe"].numel(), self.flag)
        return b["y"]

    def check(self):
        if int(self.flag):
            raise RuntimeError(f"device flag {int(self.flag)}")


def starts(new):
    return torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32, device="cuda")


def run(prompts=(100, 37, 260), steps=16, seed=0, **sizes):
    """Prompts in one call, then `steps` single tokens for each sequence. Returns the inputs, the outputs (a list per
    sequence, [prompt + steps, hidden]), the layer, and a decoding step's milliseconds."""
    layer, batch = DecoderLayer(seed=seed, **sizes), len(prompts)
    cache = Cache(batch, max(prompts) + steps, layer.hk, layer.d)
    g = torch.Generator("cuda").manual_seed(seed + 1)
    xs = [torch.randn((n + steps, layer.hidden), device="cuda", generator=g) for n in prompts]
    # prompts
    cache.lens.copy_(torch.tensor(prompts, dtype=torch.int32))
    x = torch.cat([xs[i][:n] for i, n in enumerate(prompts)])
    pos = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in prompts])
    y = layer.forward(x, pos, starts(prompts), cache, max(prompts), max(prompts), layer.buffers(len(x), batch))
    out = [[t] for t in y.split(list(prompts))]
    # single tokens: one graph, its inputs in the same buffers every step
    b, x, pos, q_start = layer.buffers(batch, batch), torch.empty((batch, layer.hidden), device="cuda"), cache.lens.clone(), starts([1] * batch)

    def step():
        pos.copy_(cache.lens)
        cache.lens.add_(1)
        layer.forward(x, pos, q_start, cache, 1, cache.max_pages * cache.page, b)
    if steps:
        keep = [t.clone() for t in (cache.lens, cache.k, cache.v, cache.k_scale, cache.v_scale)]
        x.copy_(torch.stack([xs[i][n] for i, n in enumerate(prompts)]))
        step()  # once outside: the library's one-time settings
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t, k in zip((cache.lens, cache.k, cache.v, cache.k_scale, cache.v_scale), keep):
            t.copy_(k)
    ms = 0.0
    for s in range(steps):
        x.copy_(torch.stack([xs[i][n + s] for i, n in enumerate(prompts)]))
        a, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        e.record()
        e.synchronize()
        ms += a.elapsed_time(e) / steps
        for i in range(batch):
            out[i].append(b["y"][i:i + 1].clone())
    layer.check()
    return xs, [torch.cat(o) for o in out], layer, ms


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=16)
    prompts, steps = (100, 37, 260), ap.parse_args().steps
    xs, out, layer, ms = run(prompts, steps)
    # the same tokens as prompts alone: the cache then rounds each page once
    lens = [n + steps for n in prompts]
    cache = Cache(len(lens), max(lens), layer.hk, layer.d)
    cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    pos = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in lens])
    y = layer.forward(torch.cat(xs), pos, starts(lens), cache, max(lens), max(lens), layer.buffers(sum(lens), len(lens)))
    layer.check()
    gap = max(float((a - b).abs().max()) for a, b in zip(y.split(lens), out))
    print(f"{len(prompts)} prompts of {prompts} tokens, {steps} steps of {len(prompts)} tokens at {ms:.3f} ms; "
          f"largest difference to the whole in one call {gap:.1e} of {float(y.abs().max()):.1f}")


if __name__ == "__main__":
    main()
