#!/usr/bin/env python
"""One decoder layer served with everything below 16 bits: a 4-bit paged key/value cache and E8P-coded experts.

A batch of prompts is admitted, then the sequences grow token by token.  Every step is the same five calls:

    kv4_block_tables   lengths -> block tables, slots and positions (pages from a free list)
    qk_norm_rope       norms and rotates queries and keys, and writes keys and values to the cache
    kv4_attention      attention over the cache
    qmoe_route         router
    rvq_moe_layer      the compressed experts

and the plain products around them (query/key/value and output projections, router logits) with torch.  The decode step
is captured in a CUDA graph once and replayed: its lengths, tables and free list live on the device.

With --top-blocks N it is the layer of a model for long contexts: rows are normed before the projections and the experts, a query
of a decode step attends to N blocks of its request that bounds of their keys choose, and the router scores with sigmoids, a bias
and groups of experts:

    add_rms_norm          norm of whole rows, with the residual's addition
    kv4_block_bounds      bounds of the keys of the blocks that were written to
    kv4_select_blocks     the blocks of each query token and kv head
    kv4_attention_blocks  attention over them
    qmoe_route_scored     router

    python examples/decoder_layer.py            # 2048-wide layer, 16 heads of 128, 64 experts, random weights
    python examples/decoder_layer.py --small    # a small layer, checked against a float64 restatement
    python examples/decoder_layer.py --top-blocks 8
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import decode_matvec_gb300 as Q  # noqa: E402
import synth  # noqa: E402


class Layer:
    """Weights and cache of one layer.  d_model = heads * head_dim; grouped keys; top-k SwiGLU experts."""

    def __init__(self, heads, kv_heads, head_dim, experts, d_ff, top_k, n_pages, page_size, max_blocks, max_batch, seed=0,
                 top_blocks=0):
        self.top_blocks = top_blocks
        self.heads, self.kv_heads, self.head_dim, self.top_k = heads, kv_heads, head_dim, top_k
        self.d = d = heads * head_dim
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(rows, cols):
            return (torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5).to(torch.bfloat16)
        self.w_qkv, self.w_out, self.w_router = w((heads + 2 * kv_heads) * head_dim, d), w(d, d), w(experts, d)
        self.norm_q, self.norm_k = ((1 + 0.1 * torch.randn(head_dim, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
        angle = torch.arange(page_size * max_blocks, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda", dtype=torch.float64) / head_dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        rng = np.random.default_rng(seed)

        def experts_of(rows, cols):
            return Q.RvqMatrixSet.e8p_from_host(rng.integers(0, 65536, (experts, rows, cols // 8), dtype=np.uint16),
                                                (rng.uniform(0.5, 1.5, experts * rows) * cols ** -0.5).astype(np.float16).view(np.uint16),
                                                rng.integers(0, 2, experts * rows, dtype=np.int8) * 2 - 1,
                                                rng.integers(0, 2, experts * cols, dtype=np.int8) * 2 - 1, experts, rows, cols)
        self.gate, self.up, self.down = experts_of(d_ff, d), experts_of(d_ff, d), experts_of(d, d_ff)
        self.experts, self.d_ff = experts, d_ff
        self.cache = Q.Kv4Cache.empty(n_pages, page_size, kv_heads, head_dim)
        self.table = torch.full((max_batch, max_blocks), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(n_pages, generator=g, device="cuda").int()
        self.n_free = torch.tensor([n_pages], dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(max_batch, dtype=torch.int32, device="cuda")      # tokens of each request in the cache
        if top_blocks:
            self.bounds = Q.Kv4Bounds.empty(self.cache)
            self.norm_att, self.norm_ffn = ((1 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
            self.balance = 0.02 * torch.randn(experts, generator=g, device="cuda")        # the router's bias


class Step:
    """Buffers of a step over a fixed number of tokens; call it with the layer's inputs [tokens, d_model] (bf16)."""

    def __init__(self, layer: Layer, new_tokens, max_kv: int):
        self.layer, n, B = layer, int(sum(new_tokens)), len(new_tokens)
        self.max_q, self.max_kv = max(new_tokens), max_kv
        i32 = dict(dtype=torch.int32, device="cuda")
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.new = torch.tensor(new_tokens, **i32)
        self.q_start, self.kv_len = torch.empty(B + 1, **i32), torch.empty(B, **i32)
        self.slots, self.positions = torch.empty(n, **i32), torch.empty(n, **i32)
        self.q, self.att = (torch.empty((n, layer.heads, layer.head_dim), **bf) for _ in range(2))
        self.ids, self.gates = torch.empty((n, layer.top_k), **i32), torch.empty((n, layer.top_k), dtype=torch.float32, device="cuda")
        self.ffn = torch.empty((n, layer.d), dtype=torch.float32, device="cuda")
        chosen = 0
        if layer.top_blocks:
            self.normed, self.h = (torch.empty((n, layer.d), **bf) for _ in range(2))
            self.sel = torch.empty((n, layer.kv_heads, layer.top_blocks), **i32)
            P = layer.cache.page_size
            chosen = max(Q.kv4_select_blocks_ws_size(n, layer.kv_heads, P, max_kv),
                         Q.kv4_attention_blocks_ws_size(n, layer.heads, layer.kv_heads, layer.head_dim, P, layer.top_blocks))
        self.ws = torch.empty(max(chosen, Q.kv4_attention_ws_size(B, layer.heads, layer.kv_heads, layer.head_dim, n, self.max_q, max_kv),
                                  Q.rvq_moe_layer_ws_size(layer.experts, layer.d, layer.d_ff, n, layer.top_k)), dtype=torch.uint8, device="cuda")

    def __call__(self, x):
        s, la = self, self.layer
        B = s.new.numel()
        Q.kv4_block_tables(la.lens[:B], s.new, la.free, la.n_free, la.cache.page_size, la.table[:B], s.q_start, s.kv_len, s.slots,
                           s.positions, la.n_free)
        self.seen = x                                  # what the projections see
        if la.top_blocks:
            self.seen = Q.add_rms_norm(x, la.norm_att, 1e-5, s.normed)
        Q.qk_norm_rope(self.seen @ la.w_qkv.T, la.heads, la.kv_heads, la.head_dim, la.norm_q, la.norm_k, 1e-5, la.cos_sin, s.positions, s.q,
                       cache=la.cache, slots=s.slots)
        if la.top_blocks:
            Q.kv4_block_bounds(la.cache, la.bounds, s.slots)
        if la.top_blocks and s.max_q == 1:
            Q.kv4_select_blocks(la.bounds, s.q, s.q_start, s.kv_len, la.table[:B], s.sel, s.ws, s.max_kv, first=min(1, la.top_blocks - 1))
            Q.kv4_attention_blocks(la.cache, s.q, s.q_start, s.kv_len, la.table[:B], s.sel, s.att, s.ws, la.head_dim ** -0.5)
        else:
            Q.kv4_attention(la.cache, s.q, s.q_start, s.kv_len, la.table[:B], s.att, s.ws, s.max_q, s.max_kv, la.head_dim ** -0.5)
        la.lens[:B].copy_(s.kv_len)
        if la.top_blocks:
            normed = torch.empty_like(s.h)
            Q.add_rms_norm(s.att.view(-1, la.d) @ la.w_out.T, la.norm_ffn, 1e-5, normed, residual=x, residual_out=s.h)
            Q.qmoe_route_scored(normed @ la.w_router.T, la.top_k, s.ids, s.gates, sigmoid=True, bias=la.balance, n_groups=4, top_groups=2,
                                group_best=min(2, la.experts // 4), renormalise=True, scale=1.5)
            Q.rvq_moe_layer(la.gate, la.up, la.down, normed, s.ids, s.gates, s.ffn, s.ws)
            return (s.h + s.ffn).to(torch.bfloat16), s.h
        h = x + s.att.view(-1, la.d) @ la.w_out.T
        Q.qmoe_route((h @ la.w_router.T).float(), la.top_k, s.ids, s.gates)
        Q.rvq_moe_layer(la.gate, la.up, la.down, h, s.ids, s.gates, s.ffn, s.ws)
        return (h + s.ffn).to(torch.bfloat16), h


def reference_attention(layer: Layer, xs):
    """Float64 attention output (before the projection) of sequences xs (bf16 [len, d]), from the definition: keys and values
    are rounded to bf16 and then to 4 bits, each query sees the tokens up to its own."""
    from oracle import kv4 as K
    hq, hkv, D = layer.heads, layer.kv_heads, layer.head_dim
    out = []
    for x in xs:
        # the projection as torch rounds it is an input of the attention, not a part of what is checked
        qkv = (x @ layer.w_qkv.T).double().cpu().numpy().reshape(len(x), hq + 2 * hkv, D)
        cs, pos = layer.cos_sin.double().cpu().numpy(), np.arange(len(x))
        q, k = (K.bf16_round(K.norm_rope(p, w.double().cpu().numpy(), 1e-5, cs, pos, False))
                for p, w in ((qkv[:, :hq], layer.norm_q), (qkv[:, hq:hq + hkv], layer.norm_k)))
        k, v = (K.dequantise(*K.quantise(t)).transpose(1, 0, 2) for t in (k, qkv[:, hq + hkv:]))
        out.append(K.attention(q, [0, len(x)], [k], [v], D ** -0.5)[0])
    return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--small", action="store_true")
    ap.add_argument("--steps", type=int, default=None)
    ap.add_argument("--top-blocks", type=int, default=0, help="blocks that a query of a decode step attends to (0: all, the plain layer)")
    a = ap.parse_args(argv)
    if a.small:
        layer, prompts, steps = Layer(4, 2, 64, 4, 256, 2, n_pages=64, page_size=16, max_blocks=16, max_batch=3, top_blocks=a.top_blocks), [70, 1, 33], 8
    else:
        layer, prompts, steps = Layer(16, 16, 128, 64, 1024, 8, n_pages=2048, page_size=64, max_blocks=32, max_batch=32, top_blocks=a.top_blocks), [900 + 17 * i for i in range(32)], 64
    steps = a.steps or steps
    B, cap = len(prompts), max(prompts) + steps
    rng = np.random.default_rng(1)

    def tokens(n):
        return torch.from_numpy(synth.activations_bf16(int(rng.integers(1 << 30)), n, layer.d).view(np.int16).copy()).cuda().view(torch.bfloat16)
    xs = tokens(sum(prompts))
    first = Step(layer, prompts, cap)
    first(xs)
    att = [list(x) for x in first.att.split(prompts)]
    seen = [list(x) for x in first.seen.split(prompts)]

    step, x = Step(layer, [1] * B, cap), tokens(B)
    lens, n_free = layer.lens.clone(), layer.n_free.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(x)                                    # warm up (cuBLAS); its token is taken back
        layer.lens.copy_(lens), layer.n_free.copy_(n_free)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(x)
    torch.cuda.current_stream().wait_stream(stream)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps):
        if a.small:
            x.copy_(tokens(B))
        graph.replay()
        if a.small:
            for b in range(B):
                att[b].append(step.att[b].clone())
                seen[b].append(step.seen[b].clone())
    end.record()
    assert Q.qmoe_check_status() == Q.QMOE_OK, Q.qmoe_last_error()
    print(f"{B} requests, {steps} decode steps: {begin.elapsed_time(end) / steps * 1e3:.0f} us a step, "
          f"cache {layer.cache.pages.numel() / 1e6:.0f} MB, {int(layer.n_free.item())} pages free")
    if a.small:
        worst = 0.0
        for got, ref in zip(att, reference_attention(layer, [torch.stack(s) for s in seen])):
            worst = max(worst, float(np.linalg.norm(torch.stack(got).double().cpu().numpy() - ref) / np.linalg.norm(ref)))
        print(f"attention against float64: relative error {worst:.1e}")
        return worst
    return None


if __name__ == "__main__":
    main()
