"""Definitions of the decode-step operators in float64 (numpy, plain loops over
requests and heads), with the sums of magnitudes that rounding bounds need.

  w4_matvec        products with 4-bit weights and group scales
  rotate / append  per-head RMS norm, rotation, append to a paged cache
  append_axes      the same with positions of several axes
  attention_weights  the weights that cached tokens get from it
  evict            eviction from a paged cache by scores
  tree_attention   attention of drafted tokens over a paged cache
"""
from __future__ import annotations

import numpy as np


def w4_weights(codes, scales, zeros, group):
    """Dense float64 weights [h_out, h_in] of packed codes [h_out, h_in/2] (low half first)."""
    c = np.asarray(codes, np.uint8)
    q = np.empty((c.shape[0], 2 * c.shape[1]), np.float64)
    q[:, 0::2] = c & 15
    q[:, 1::2] = c >> 4
    z = np.full(scales.shape, 8.0) if zeros is None else np.asarray(zeros, np.float64)
    return (q - np.repeat(z, group, 1)) * np.repeat(np.asarray(scales, np.float64), group, 1)


def w4_matvec(x, codes, scales, zeros, group):
    """(y, sum of |terms|), both [T, h_out]."""
    w = w4_weights(codes, scales, zeros, group)
    x = np.asarray(x, np.float64)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def rotate(x, cos, sin, interleaved):
    """x [..., d]; the first 2 * len(cos) elements are rotated pair by pair."""
    y = np.array(x, np.float64)
    half = len(cos)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        y[..., a] = x[..., a] * cos[i] - x[..., b] * sin[i]
        y[..., b] = x[..., a] * sin[i] + x[..., b] * cos[i]
    return y


def rms_norm(x, weight, eps):
    x = np.asarray(x, np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def append(q, k, v, positions, slots, cos_sin, rot, interleaved, q_norm, k_norm, eps, k_pages, v_pages):
    """q [T, n_q, d], k and v [T, n_kv, d]; returns (q_out, k_pages, v_pages) with the pages copied."""
    T, page = len(slots), k_pages.shape[2]
    k_pages, v_pages = np.array(k_pages, np.float64), np.array(v_pages, np.float64)
    q_out = np.empty(q.shape, np.float64)
    half = rot // 2
    for t in range(T):
        row = np.asarray(cos_sin[positions[t]], np.float64) if rot else np.zeros(0)
        c, s = row[:half], row[half:]
        q_out[t] = rotate(rms_norm(q[t], q_norm, eps), c, s, interleaved)
        if slots[t] < 0:
            continue
        p, off = divmod(int(slots[t]), page)
        k_pages[p, :, off] = rotate(rms_norm(k[t], k_norm, eps), c, s, interleaved)
        v_pages[p, :, off] = v[t]
    return q_out, k_pages, v_pages


def append_axes(q, k, v, positions, pair_axis, slots, cos_sin, rot, interleaved, q_norm, k_norm, eps, k_pages, v_pages):
    """append() with positions [T, axes]: pair i of token t turns by the table's row positions[t][pair_axis[i]]."""
    half = rot // 2
    rows = np.empty((len(slots), 2 * half))
    for t in range(len(slots)):
        for i in range(half):
            rows[t, i], rows[t, half + i] = (cos_sin[positions[t][pair_axis[i]]][x] for x in (i, half + i))
    return append(q, k, v, np.arange(len(slots)), slots, rows, rot, interleaved, q_norm, k_norm, eps, k_pages, v_pages)


def visible(n, kv_len, mask_rows):
    """[n, kv_len] truth values; mask_rows [n, n] truth values, or None for a causal chain."""
    see = np.ones((n, kv_len), bool)
    drafted = np.tril(np.ones((n, n), bool)) if mask_rows is None else np.asarray(mask_rows, bool)
    see[:, kv_len - n:] = drafted
    return see


def tree_attention(q, k_pages, v_pages, starts, lens, table, masks, scale):
    """q [T, n_q, d]; masks: per request [n, n] truth values or None.  Returns (out [T, n_q, d], sum of p |v|
    [T, n_q, d], largest scale * sum |q k| [T, n_q])."""
    q = np.asarray(q, np.float64)
    T, n_q, d = q.shape
    n_kv, page = k_pages.shape[1], k_pages.shape[2]
    out, mag, big = np.zeros((T, n_q, d)), np.zeros((T, n_q, d)), np.zeros((T, n_q))
    for s in range(len(lens)):
        b, e, length = int(starts[s]), int(starts[s + 1]), int(lens[s])
        n = e - b
        if n == 0 or length == 0:
            continue
        ids = np.asarray(table[s][: -(-length // page)])
        see = visible(n, length, None if masks is None else masks[s])
        for h in range(n_kv):
            k = np.asarray(k_pages[ids, h], np.float64).reshape(-1, d)[:length]
            v = np.asarray(v_pages[ids, h], np.float64).reshape(-1, d)[:length]
            for hq in range(h * (n_q // n_kv), (h + 1) * (n_q // n_kv)):
                for i in range(n):
                    on = np.flatnonzero(see[i])
                    if not len(on):
                        continue
                    sc = scale * (k[on] @ q[b + i, hq])
                    p = np.exp(sc - sc.max())
                    p /= p.sum()
                    out[b + i, hq] = p @ v[on]
                    mag[b + i, hq] = p @ np.abs(v[on])
                    big[b + i, hq] = (scale * (np.abs(k[on]) @ np.abs(q[b + i, hq]))).max()
    return out, mag, big


def attention_weights(q, k_pages, starts, lens, table, masks, scale, weights, decay):
    """weights [n_pages, n_kv, page] after the attention of q [T, n_q, d]; also, of the same shape, the sum of what was
    added and that sum with each term times its row's largest scale * sum |q k|."""
    q = np.asarray(q, np.float64)
    n_q, n_kv, page = q.shape[1], k_pages.shape[1], k_pages.shape[2]
    new, gain, loaded = np.array(weights, np.float64), np.zeros(weights.shape), np.zeros(weights.shape)
    for s in range(len(lens)):
        b, e, length = int(starts[s]), int(starts[s + 1]), int(lens[s])
        n = e - b
        if n == 0:
            continue
        ids = np.asarray(table[s][: -(-length // page)])
        see = visible(n, length, None if masks is None else masks[s])
        for h in range(n_kv):
            k = np.asarray(k_pages[ids, h], np.float64).reshape(len(ids) * page, -1)[:length]
            total, load = np.zeros(length), np.zeros(length)
            for hq in range(h * (n_q // n_kv), (h + 1) * (n_q // n_kv)):
                for i in range(n):
                    on = np.flatnonzero(see[i])
                    if not len(on):
                        continue
                    sc = scale * (k[on] @ q[b + i, hq])
                    p = np.exp(sc - sc.max())
                    p /= p.sum()
                    total[on] += p
                    load[on] += p * (scale * (np.abs(k[on]) @ np.abs(q[b + i, hq]))).max()
            for c in range(length):
                at = (ids[c // page], h, c % page)
                new[at] = total[c] + (decay * new[at] if c < length - n and decay else 0.0)
                gain[at], loaded[at] = total[c], load[c]
    return new, gain, loaded


def evict(planes, scores, lens, table, keep, first, recent):
    """planes: arrays [n_pages, n_kv, page, ..] that move with the tokens; scores [n_pages, n_kv, page].  Returns (planes
    moved, per request None or the kept indices [n_kv, keep[s]], new lengths)."""
    planes = [np.array(p) for p in planes]
    n_kv, page = scores.shape[1], scores.shape[2]
    kept, new_lens = [None] * len(lens), np.array(lens)
    for s, length in enumerate(np.asarray(lens).tolist()):
        budget = int(keep[s])
        if budget < 0 or length <= budget:
            continue
        last = min(recent, budget)
        begin = min(first, budget - last)
        slot = [(int(table[s][c // page]), c % page) for c in range(length)]
        rows = []
        for h in range(n_kv):
            def value(c):
                f = float(scores[slot[c][0], h, slot[c][1]])
                return (f == f, f if f == f else 0.0)      # a NaN is below everything
            middle = sorted(range(begin, length - last), key=lambda c: (*(-x for x in value(c)), c))
            chosen = sorted([*range(begin), *middle[: budget - begin - last], *range(length - last, length)])
            for p in planes:
                old = [np.array(p[slot[c][0], h, slot[c][1]]) for c in chosen]
                for j, o in enumerate(old):
                    p[slot[j][0], h, slot[j][1]] = o
            rows.append(chosen)
        kept[s] = np.array(rows, np.int64).reshape(n_kv, budget)
        new_lens[s] = budget
    return planes, kept, new_lens
