#!/usr/bin/env python3
"""A stream of images and text through one attention block whose cache stays bounded.

Every request gets an image now and then, as a chunk of patches, and decodes text in between:

    q, k, v = x W4^T + adapter       lora_w4_matvec, then lora_bgmv
    norm, rotate, append             lora_kv_append_axes: time, height and width of a patch; text has one position on all axes
    attention, weights kept          lora_tree_attention_weights
    output projection + adapter      lora_w4_matvec, then lora_bgmv
    eviction                         lora_kv_evict, when a request is past its budget by more than a slack

    python examples/bounded_cache.py [--requests 16] [--budget 1024] [--slack 128] [--images 6] [--steps 64]

prints how long a decode step and an eviction take.  Weights, adapters and inputs are random.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from decode_attention import L, AttentionBlock  # noqa: E402


class BoundedBlock(AttentionBlock):
    """The block of decode_attention.py with three-axis positions and a cache of at most `budget` tokens a request after an
    eviction: the first `first`, the last `recent`, and of the others, head by head, those that got the most attention."""

    def __init__(self, requests, budget, slack, chunk, first=4, recent=64, decay=0.99, page=16, **kw):
        self.requests, self.budget, self.slack, self.first, self.recent, self.decay = requests, budget, slack, first, recent, decay
        self.longest = budget + slack + chunk
        self.max_pages = -(-self.longest // page)
        super().__init__(page=page, n_pages=requests * self.max_pages, max_tokens=requests * chunk, **kw)
        half = self.d // 2
        self.pair_axis = bytes(np.searchsorted(np.round(np.array([0.2, 0.6, 1.0]) * half), np.arange(half), side="right").tolist())
        self.weights = torch.zeros(requests * self.max_pages, self.n_kv, page, device="cuda")
        ids = torch.randperm(requests * self.max_pages, dtype=torch.int32)
        self.table = ids.view(requests, self.max_pages).cuda()
        self.held = np.zeros(requests, np.int64)                 # cached tokens of each request
        self.kept = torch.empty(requests, self.n_kv, budget, dtype=torch.int32, device="cuda")
        self.new_lens = torch.empty(requests, dtype=torch.int32, device="cuda")
        self.budgets = torch.full((requests,), budget, dtype=torch.int32, device="cuda")
        size = max(L.lora_tree_attention_weights_workspace_size(self.kv, self.n_q, requests, t, self.max_pages)
                   for t in (requests, requests * chunk))
        self.workspace = torch.empty(size, dtype=torch.uint8, device="cuda")

    def tables(self, new):
        """Slots and lengths of a step that adds new[s] tokens to request s."""
        new = np.asarray(new)
        request = np.repeat(np.arange(self.requests), new)
        at = np.concatenate([h + np.arange(n) for h, n in zip(self.held, new)]).astype(np.int64)
        page = torch.from_numpy(at // self.page).cuda()
        slots = self.table[torch.from_numpy(request).cuda(), page].long() * self.page + torch.from_numpy(at % self.page).cuda()
        starts = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
        return dict(slots=slots, starts=starts, lens=torch.from_numpy((self.held + new).astype(np.int32)).cuda())

    def step(self, x, token_adapter, positions, slots, starts, lens):
        """x [T, hidden], positions [T, 3]: the block's output [T, hidden]; the caller counts the tokens (`held`)."""
        T = x.shape[0]
        q, k, v = (self.project(n, x, token_adapter) for n in ("q", "k", "v"))
        L.lora_kv_append_axes(self.kv, q, k, v, T, self.n_q, positions, 3, self.pair_axis, slots, self.cos_sin, self.max_position, self.d,
                              False, q, q_norm=self.q_norm, k_norm=self.k_norm)
        out = self.attended[:T]
        L.lora_tree_attention_weights(self.kv, self.weights, self.decay, q, self.n_q, starts, self.requests, T, lens, self.table,
                                      self.max_pages, None, 0, 1 / math.sqrt(self.d), out, self.workspace)
        return self.project("o", out, token_adapter)

    def evict(self):
        """Cuts the requests that are past their budget by more than the slack."""
        over = self.held > self.budget + self.slack
        if not over.any():
            return False
        lens = torch.from_numpy(self.held.astype(np.int32)).cuda()
        self.budgets.copy_(torch.from_numpy(np.where(over, self.budget, -1).astype(np.int32)))
        L.lora_kv_evict(self.kv, self.weights, self.weights, self.requests, lens, self.table, self.max_pages, self.budgets, self.first,
                        self.recent, self.kept, self.budget, self.new_lens)
        self.held = np.where(over, self.budget, self.held)
        return True


def image(begin, side):
    """Positions of a side x side image that begins at `begin`: one time, rows, columns."""
    i = np.arange(side * side)
    return np.stack([np.full(side * side, begin), begin + i // side, begin + i % side], 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--budget", type=int, default=1024)
    ap.add_argument("--slack", type=int, default=128)
    ap.add_argument("--images", type=int, default=6)
    ap.add_argument("--side", type=int, default=20)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    S = a.requests
    block = BoundedBlock(S, a.budget, a.slack, a.side * a.side)
    adapter = torch.arange(S, device="cuda", dtype=torch.int32) % 16
    now = np.zeros(S, np.int64)                                  # the next position of each request
    times = {"step": [], "eviction": []}

    def timed(what, f):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        done = f()
        end.record()
        if done is not False:
            times[what].append((begin, end))

    for _ in range(a.images):
        n = a.side * a.side
        positions = torch.from_numpy(np.concatenate([image(p, a.side) for p in now]).astype(np.int32)).cuda()
        block.step(torch.randn(S * n, block.hidden, device="cuda").bfloat16(), adapter.repeat_interleave(n), positions, **block.tables([n] * S))
        block.held += n
        now += a.side
        timed("eviction", block.evict)
        for _ in range(a.steps):
            positions = torch.from_numpy(np.repeat(now[:, None], 3, 1).astype(np.int32)).cuda()
            x, tables = torch.randn(S, block.hidden, device="cuda").bfloat16(), block.tables([1] * S)
            timed("step", lambda: block.step(x, adapter, positions, **tables))
            block.held += 1
            now += 1
            timed("eviction", block.evict)
    torch.cuda.synchronize()
    if int(block.status):
        raise SystemExit(f"device status {int(block.status)}")
    print(f"{S} requests, {int(now[0])} positions and {a.images * (a.side * a.side + a.steps)} tokens each, at most {block.longest} cached")
    for what, pairs in times.items():
        if pairs:
            us = sorted(b.elapsed_time(e) * 1e3 for b, e in pairs)
            print(f"{what}: {us[len(us) // 2]:.1f} us ({len(us)} of them)")
    block.close()


if __name__ == "__main__":
    main()
