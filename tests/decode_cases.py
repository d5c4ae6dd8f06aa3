"""Seeded cases of the decode-step operators for the tests: host arrays (float32 holding values exact in the
type), their device copies, and the rounding bounds of the kernels' outputs.

Bounds, from the arithmetic (u = 2^-24 fp32, a store to bf16 adds 2^-9 of the value):
* products with 4-bit weights: the codes less zeros are exact in bf16, fp32 activations enter as up to three bf16
  parts (24 bits), sums are fp32.  A sum of K terms taken 16 at a time rounds K/16 + 16 times, each by at most
  2u (the tensor cores truncate) of the sum of magnitudes, and the scaling and the sum over groups once more each.
* norm and rotation: fewer than 2 log2(d) + 16 roundings of the largest magnitude of a head, and the square root's.
* attention: a score is off by at most (d + 4) u of scale * sum |q k|, so each probability by that factor of
  itself (twice: numerator and denominator), exp by 2^-20 at most, the sums by (log-many partial sums and) 2^-18;
  for a bf16 cache each probability is rounded to bf16 (2^-8 with the normaliser's share) before the second product.
"""
import numpy as np
import torch

from segmented_gathered_rank_gb300 import inputs as I

U = 2.0 ** -24


def store(a, dtype):
    a = np.asarray(a, np.float32)
    return I.round_to_bf16(a) if dtype == I.BF16 else a


def w4_case(seed, dtype, T, h_in, h_out, group, zeros):
    rng = np.random.default_rng(seed)
    x = store(rng.normal(0, 1, (T, h_in)), dtype)
    codes = rng.integers(0, 256, (h_out, h_in // 2), dtype=np.uint8)
    scales = I.round_to_bf16(rng.uniform(0.002, 0.01, (h_out, h_in // group)).astype(np.float32))
    z = rng.integers(0, 16, scales.shape, dtype=np.uint8) if zeros else None
    return x, codes, scales, z


def w4_bound(ref, mag, h_in, group, dtype):
    return (2.0 ** -8 if dtype == I.BF16 else 2 * U) * np.abs(ref) + 2 * U * (h_in / 16 + 16 + h_in / group) * mag + 1e-30


def tree_masks(rng, n, kind):
    """[n, n] truth values: a random tree's ancestors, a chain (None is the kernel's own), or random bits."""
    see = np.zeros((n, n), bool)
    if kind == "tree":
        for i in range(n):
            if i:
                see[i] = see[rng.integers(max(0, i - 6), i)]
            see[i, i] = True
    elif kind == "random":
        see = rng.random((n, n)) < 0.3
    return see


def pack_masks(masks, words):
    rows = []
    for m in masks:
        wide = np.zeros((len(m), words * 64), bool)
        wide[:, : min(m.shape[1], words * 64)] = m[:, : words * 64]
        rows.append(np.packbits(wide, axis=1, bitorder="little"))
    return np.ascontiguousarray(np.concatenate(rows)).view("<i8")


class Attention:
    """requests: list of (drafted n, cached length with the drafted)."""

    def __init__(self, seed, dtype, requests, n_q, n_kv, d, page, mask=None, words=None, garbage=np.nan, scale=None):
        rng = np.random.default_rng(seed)
        self.dtype, self.n_q, self.n_kv, self.d, self.page = dtype, n_q, n_kv, d, page
        self.S = len(requests)
        ns = [r[0] for r in requests]
        self.lens = np.array([r[1] for r in requests], np.int32)
        self.starts = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        self.T = int(self.starts[-1])
        self.max_pages = max(1, int(max(-(-self.lens // page))))
        used = [-(-int(n) // page) for n in self.lens]
        self.n_pages = sum(used) + 2
        ids = rng.permutation(self.n_pages)
        self.table = np.full((self.S, self.max_pages), -1, np.int32)
        self.k = np.full((self.n_pages, n_kv, page, d), garbage, np.float32)
        self.v = np.full((self.n_pages, n_kv, page, d), garbage, np.float32)
        at = 0
        for s, count in enumerate(used):
            self.table[s, :count] = ids[at: at + count]
            at += count
            for c in range(count):       # only slots that hold tokens get values
                fill = min(page, int(self.lens[s]) - c * page)
                for pages in (self.k, self.v):
                    pages[self.table[s, c], :, :fill] = store(rng.normal(0, 1, (n_kv, fill, d)), dtype)
        self.q = store(rng.normal(0, 1, (self.T, n_q, d)), dtype)
        self.scale = float(np.float32(d ** -0.5 if scale is None else scale))
        self.masks, self.bits, self.words = None, None, 1
        if mask is not None:
            self.masks = [mask(rng, n) if callable(mask) else tree_masks(rng, n, mask) for n in ns]
            self.words = words or max(1, (max(ns) + 63) // 64)
            self.bits = pack_masks(self.masks, self.words)

    def bound(self, ref, mag, big):
        score = (self.d + 4) * U * big[..., None]
        p = 2.0 ** -8 if self.dtype == I.BF16 else 0.0
        return (2.0 ** -8 if self.dtype == I.BF16 else 2 * U) * np.abs(ref) + (2 * score + 2.0 ** -18 + p) * mag + 1e-30


def device(a, dtype):
    from segmented_gathered_rank_gb300 import harness as H
    if dtype == I.BF16:      # bf16_bits refuses NaN payloads; to_device keeps the rest exact
        t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()
        return t.to(torch.bfloat16)
    return H.to_device(a, dtype)
