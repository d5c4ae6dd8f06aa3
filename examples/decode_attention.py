#!/usr/bin/env python3
"""Decode steps of one attention block under many adapters, on the library's calls.

Each request adds one token a step, or verifies a small tree of drafted ones:

    q, k, v = x W4^T + adapter       lora_w4_matvec, then lora_bgmv
    norm, rotate, append             lora_kv_append
    attention over the paged cache   lora_tree_attention
    output projection + adapter      lora_w4_matvec, then lora_bgmv

    python examples/decode_attention.py [--requests 32] [--drafts 8] [--context 2000] [--steps 20]

captures a step in a CUDA graph, replays it and prints the time of a step.
Weights, adapters and the context are random.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from segmented_gathered_rank_gb300 import inputs as I  # noqa: E402
from segmented_gathered_rank_gb300 import lora as L  # noqa: E402


class Projection:
    """A base weight in 4 bits; its adapters are matrix ``index`` of the block's pool."""

    def __init__(self, rng, index, h_in, h_out, group=128):
        self.index, self.h_in, self.h_out, self.group = index, h_in, h_out, group
        self.codes_host = rng.integers(0, 256, (h_out, h_in // 2), dtype=np.uint8)
        self.scales_host = I.round_to_bf16(rng.uniform(0.1, 0.3, (h_out, h_in // group)).astype(np.float32) / math.sqrt(h_in))
        self.zeros_host = rng.integers(6, 10, self.scales_host.shape, dtype=np.uint8)
        self.codes = torch.from_numpy(self.codes_host).cuda()
        self.scales = torch.from_numpy(self.scales_host).cuda().to(torch.bfloat16)
        self.zeros = torch.from_numpy(self.zeros_host).cuda()


class AttentionBlock:
    def __init__(self, hidden=4096, n_q=32, n_kv=8, head_dim=128, adapters=16, rank=16, page=16, n_pages=4096, max_tokens=512,
                 max_position=1 << 16, seed=0):
        rng = np.random.default_rng(seed)
        self.hidden, self.n_q, self.n_kv, self.d, self.page, self.max_position = hidden, n_q, n_kv, head_dim, page, max_position
        widths = {"q": (hidden, n_q * head_dim), "k": (hidden, n_kv * head_dim), "v": (hidden, n_kv * head_dim),
                  "o": (n_q * head_dim, hidden)}
        self.proj = {name: Projection(rng, i, *w) for i, (name, w) in enumerate(widths.items())}
        page_elems = max(max(w) for w in widths.values())
        self.pool = L.lora_pool_create(L.LORA_BF16, page_elems, 2 * rank * adapters * 4, rank, 4, adapters)
        self.adapters_host = {}
        for p in self.proj.values():
            for a in range(adapters):
                at = I.round_to_bf16(rng.normal(0, 1 / math.sqrt(p.h_in), (rank, p.h_in)).astype(np.float32))
                b = I.round_to_bf16(rng.normal(0, 0.3, (rank, p.h_out)).astype(np.float32))
                self.adapters_host[p.index, a] = (at, b)
                L.lora_pool_load(self.pool, a, p.index, rank, 1.0, p.h_in, p.h_out, I.bf16_bits(at), I.bf16_bits(b))
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.q_norm = (1 + 0.1 * torch.randn(head_dim, device="cuda")).bfloat16()
        self.k_norm = (1 + 0.1 * torch.randn(head_dim, device="cuda")).bfloat16()
        angle = torch.arange(max_position, dtype=torch.float64)[:, None] * \
            torch.pow(10000.0, -torch.arange(head_dim // 2, dtype=torch.float64) / (head_dim // 2))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        self.k_pages = torch.randn(n_pages, n_kv, page, head_dim, **bf16)
        self.v_pages = torch.randn(n_pages, n_kv, page, head_dim, **bf16)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.kv = L.KvPages(L.LORA_BF16, self.k_pages, self.v_pages, n_pages, page, n_kv, head_dim, status=self.status)
        self.y = {n: torch.empty(max_tokens, p.h_out, **bf16) for n, p in self.proj.items()}
        self.attended = torch.empty(max_tokens, n_q * head_dim, **bf16)
        # a graph's buffers stay where they are: the workspace for any batch of up to max_tokens
        size = max(L.lora_tree_attention_workspace_size(self.kv, n_q, s, max_tokens) for s in (1, max_tokens))
        self.workspace = torch.empty(size, dtype=torch.uint8, device="cuda")

    def close(self):
        L.lora_pool_destroy(self.pool)

    def project(self, name, x, token_adapter):
        p, T = self.proj[name], x.shape[0]
        y = self.y[name][:T]
        L.lora_w4_matvec(L.LORA_BF16, x, T, p.h_in, p.codes, p.scales, p.zeros, p.group, p.h_out, y)
        L.lora_bgmv(self.pool, p.index, x, y, token_adapter, T)
        return y

    def step(self, x, token_adapter, positions, slots, starts, lens, table, tree_mask):
        """x [T, hidden]: the block's output [T, hidden].  lens count the tokens of this step."""
        T, S = x.shape[0], lens.shape[0]
        q, k, v = (self.project(n, x, token_adapter) for n in ("q", "k", "v"))
        L.lora_kv_append(self.kv, q, k, v, T, self.n_q, positions, slots, self.cos_sin, self.max_position, self.d, False, q,
                         q_norm=self.q_norm, k_norm=self.k_norm)
        out = self.attended[:T]
        size = L.lora_tree_attention_workspace_size(self.kv, self.n_q, S, T)
        if size > self.workspace.numel():
            self.workspace = torch.empty(size, dtype=torch.uint8, device="cuda")
        L.lora_tree_attention(self.kv, q, self.n_q, starts, S, T, lens, table, table.shape[1], tree_mask,
                              0 if tree_mask is None else tree_mask.shape[1], 1 / math.sqrt(self.d), out, self.workspace)
        return self.project("o", out, token_adapter)


def batch(block, requests, drafts, context, adapters=16, seed=1):
    """Device tables of a step: every request holds about `context` tokens and drafts `drafts` (at most 64) more, a
    random tree whose nodes' positions are their depths."""
    rng = np.random.default_rng(seed)
    prefix = rng.integers(max(1, context // 2), context + 1, requests)
    lens = (prefix + drafts).astype(np.int32)
    used = -(-lens // block.page)
    table = np.full((requests, int(used.max())), -1, np.int32)
    ids = rng.permutation(block.k_pages.shape[0])
    if used.sum() > len(ids):
        raise ValueError("the cache is too small for this batch")
    for s, at in enumerate(np.cumsum(used) - used):
        table[s, : used[s]] = ids[at: at + used[s]]
    T = requests * drafts
    bits, depth = np.zeros((T, 1), np.uint64), np.zeros(T, np.int64)
    for t in range(T):
        i = t % drafts
        parent = t - 1 - int(rng.integers(0, min(i, 4))) if i else -1
        bits[t, 0] = (bits[parent, 0] if i else np.uint64(0)) | np.uint64(1 << i)
        depth[t] = depth[parent] + 1 if i else 0
    request = np.repeat(np.arange(requests), drafts)
    at = prefix[request] + np.arange(T) % drafts
    cuda = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a, dt)).cuda()  # noqa: E731
    return dict(token_adapter=cuda(rng.integers(0, adapters, requests)[request], np.int32), positions=cuda(prefix[request] + depth, np.int32),
                slots=cuda(table[request, at // block.page].astype(np.int64) * block.page + at % block.page, np.int64),
                starts=cuda(np.arange(requests + 1) * drafts, np.int32), lens=cuda(lens, np.int32), table=cuda(table, np.int32),
                tree_mask=cuda(bits.view(np.int64), np.int64))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=32)
    ap.add_argument("--drafts", type=int, default=8)
    ap.add_argument("--context", type=int, default=2000)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    T = a.requests * a.drafts
    block = AttentionBlock(n_pages=a.requests * (a.context + a.drafts + 16) // 16 + 16, max_tokens=T)
    tables = batch(block, a.requests, a.drafts, a.context)
    x = torch.randn(T, block.hidden, device="cuda").bfloat16()
    block.step(x, **tables)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x, **tables)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if int(block.status) or not bool(torch.isfinite(y.float()).all()):
        raise SystemExit(f"device status {int(block.status)}")
    print(f"{a.requests} requests x {a.drafts} drafted tokens over about {a.context}: "
          f"{begin.elapsed_time(end) / a.steps * 1e3:.1f} us a step")
    block.close()


if __name__ == "__main__":
    main()
