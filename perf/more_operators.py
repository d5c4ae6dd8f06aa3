"""Cases, plain forms and exact results of the operators of a cache that stays bounded.

A long stream of text, images and video passes through one attention block:
its tokens are appended at positions with several axes
(``lora_kv_append_axes``), attention sums up the weight that each cached token
gets (``lora_tree_attention_weights``), and the tokens with the least are
evicted (``lora_kv_evict``).

``own`` false: ``run`` computes the formulas with elementary torch operations
in 32 bits, rounded once.  ``own`` true: it calls the library.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
_DTYPES = {BF16: torch.bfloat16, F32: torch.float32}
_ESIZE = {BF16: 2, F32: 4}


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # The next text token after an image: one append, three axes in sections of the head.
        dict(name="axes_1", op="axes", dtype=BF16, T=1, n_q=32, n_kv=8, d=128, rot=128, page=16, axes=3, cycle=False,
             interleaved=False, norm=True, fused=True, max_pos=8192),
        # A video prompt of 8192 patches, axes taken in turn by the pairs, one fused qkv matrix.
        dict(name="axes_8192", op="axes", dtype=BF16, T=8192, n_q=32, n_kv=8, d=128, rot=128, page=64, axes=3, cycle=True,
             interleaved=False, norm=True, fused=True, max_pos=8192),
        # Odd everything: two axes on 20 of 80 elements, neighbours paired, 7 query heads on one kv head, fp32.
        dict(name="axes_odd_f32", op="axes", dtype=F32, T=333, n_q=7, n_kv=1, d=80, rot=20, page=8, axes=2, cycle=False,
             interleaved=True, norm=True, fused=False, max_pos=2048),
        # One request decodes one token over a short context: the smallest attention.
        dict(name="weigh_1", op="weigh", dtype=BF16, S=1, n=1, max_len=777, n_q=32, n_kv=8, d=128, page=16, mask="chain",
             padded=False, decay=1.0),
        # A decode batch: 128 requests of very different lengths, one token each, older weight fading.
        dict(name="weigh_decode_128", op="weigh", dtype=BF16, S=128, n=1, max_len=8192, n_q=32, n_kv=8, d=128, page=16,
             mask="chain", padded=False, decay=0.98),
        # Two requests decode over very long contexts.
        dict(name="weigh_long_2", op="weigh", dtype=BF16, S=2, n=1, max_len=131072, n_q=32, n_kv=8, d=128, page=16,
             mask="chain", padded=False, decay=1.0),
        # The last 64 tokens of eight prompts, whose weights alone decide what is kept of them.
        dict(name="weigh_window_64", op="weigh", dtype=BF16, S=8, n=64, max_len=16384, n_q=32, n_kv=8, d=128, page=64,
             mask="chain", padded=False, decay=0.0),
        # fp32, an odd head width, five requests with padded trees, some of them without any context.
        dict(name="weigh_odd_f32", op="weigh", dtype=F32, S=5, n=7, max_len=300, n_q=6, n_kv=2, d=80, page=8, mask="tree",
             padded=True, decay=0.5),
        # One request has gone 64 tokens past its budget.
        dict(name="evict_1", op="evict", dtype=BF16, S=1, max_len=1088, keep=1024, first=4, recent=128, n_kv=8, d=128, page=16,
             ragged=False, ties=False),
        # A batch of 64 requests, each up to 256 tokens past its budget; the shorter ones keep everything.
        dict(name="evict_64", op="evict", dtype=BF16, S=64, max_len=4352, keep=4096, first=4, recent=512, n_kv=8, d=128, page=16,
             ragged=True, ties=False),
        # Four long prompts are cut to a sixteenth, many of their tokens with equal weights.
        dict(name="evict_prompt_4", op="evict", dtype=BF16, S=4, max_len=32768, keep=2048, first=16, recent=64, n_kv=8, d=128,
             page=64, ragged=False, ties=True),
        # fp32, an odd head width, small pages, budgets that are no multiple of a page.
        dict(name="evict_odd_f32", op="evict", dtype=F32, S=5, max_len=999, keep=333, first=1, recent=17, n_kv=3, d=80, page=8,
             ragged=True, ties=True),
    ]


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm, off the grid of 1024 that listed cases lie on."""
    v = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return v - 1 if v % 1024 == 0 else v


def draw(rng):
    """One more case: T and lengths over their logarithm; costs at most the largest listed case of its operator."""
    op = rng.choice(["axes", "weigh", "evict"])
    cap = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        n_kv = rng.choice([1, 2, 4, 8])
        case = dict(op=op, dtype=rng.choice([BF16, BF16, BF16, F32]), n_kv=n_kv, d=rng.choice([64, 80, 112, 128, 128, 256]),
                    page=rng.choice([1, 8, 16, 32, 64, 128]))
        if op != "evict":
            case["n_q"] = n_kv * rng.choice([1, 2, 4, 7, 8])
        if op == "axes":
            case["rot"] = case["d"] if rng.random() < 0.6 else 2 * rng.randint(2, case["d"] // 2)
            case.update(T=_spread(rng, 1, 8192), axes=rng.choice([2, 3, 3, 4]), cycle=rng.random() < 0.5, interleaved=rng.random() < 0.4,
                        norm=rng.random() < 0.6, fused=rng.random() < 0.5, max_pos=_spread(rng, 512, 131072))
            if case["fused"] and (case["n_q"] + 2 * n_kv) * case["d"] % 1024 == 0:
                case["fused"] = False
        elif op == "weigh":
            n = rng.choice([1, 1, _spread(rng, 1, 128)])
            case.update(S=_spread(rng, 1, 128), n=n, max_len=max(n, _spread(rng, 16, 131072)),
                        mask=rng.choice(["tree", "chain"]) if n > 1 else "chain", padded=n > 1 and rng.random() < 0.4,
                        decay=rng.choice([0.0, 0.5, 0.98, 1.0, 1.0]))
            plain = case["S"] * case["n_q"] * n * case["max_len"] + case["S"] * case["max_len"] * n_kv * case["d"]
            if plain > 2 ** 31:     # the plain form pads every request to the longest one
                continue
        else:
            top = _spread(rng, 16, 65536)
            keep = max(1, min(top - 1, int(top * rng.choice([0.05, 0.25, 0.5, 0.9, 0.97]))))
            case.update(S=_spread(rng, 1, 128), max_len=top, keep=keep, first=rng.randint(0, min(16, keep)),
                        recent=int(keep * rng.uniform(0, 0.5)), ragged=rng.random() < 0.5, ties=rng.random() < 0.4)
            if case["S"] * top * n_kv * case["d"] * 2 * _ESIZE[case["dtype"]] > 8e9:       # the caches
                continue
        if _cost(case) <= cap:
            return case


def _lengths(case):
    """Drafted tokens and cached tokens (the drafted ones among them) of each request: ragged, the first request the
    longest; with "padded", some requests hold no context before their drafts and some draft nothing."""
    S, n, top = case["S"], case["n"], case["max_len"]
    rng = np.random.default_rng([S, n, top])
    drafts = np.full(S, n) if n == 1 else rng.integers((n + 1) // 2, n + 1, S)
    context = np.floor((top - n) * rng.random(S) ** 1.5).astype(np.int64)
    if case["padded"]:
        context[rng.random(S) < 0.3] = 0
        drafts[rng.random(S) < 0.2] = 0
    drafts[0], context[0] = n, top - n
    return drafts.astype(np.int64), context + drafts


def _visible(case):
    """Per drafted token (requests in order) the drafted tokens of its request that it sees, as truth values
    [T, n]: its ancestors and itself in a random tree, or (chain) every one up to itself.  With "padded" the
    last quarter of a tree's tokens are padding that sees no drafted token."""
    drafts, _ = _lengths(case)
    n = case["n"]
    see = np.zeros((case["S"], n, n), bool)
    rng = np.random.default_rng([case["S"], n, 7])
    parent = np.maximum(np.arange(n) - 1 - (rng.random(n) * np.minimum(np.arange(n), 8)).astype(np.int64), 0)
    for i in range(n):
        if case["mask"] == "chain":
            see[:, i, : i + 1] = True
        else:
            see[:, i] = see[:, parent[i]] if i else False
            see[:, i, i] = True
    if case["padded"] and case["mask"] == "tree":
        see[np.arange(n)[None, :] >= np.ceil(0.75 * drafts)[:, None]] = False
    return see[np.arange(n)[None, :] < drafts[:, None]], drafts


def _evicted_lengths(case):
    """Cached tokens of each request: all at the largest, or ragged from nothing to it."""
    rng = np.random.default_rng([case["S"], case["max_len"], 5])
    lens = np.full(case["S"], case["max_len"])
    if case["ragged"]:
        lens = np.floor(case["max_len"] * (1 - rng.random(case["S"]) ** 2)).astype(np.int64)
        lens[0] = case["max_len"]
    return lens.astype(np.int64)


def _pair_axes(case):
    """The axis of each pair: in turn, or one section an axis, the first (time) half as long as the others."""
    half, n = case["rot"] // 2, case["axes"]
    if case["cycle"]:
        return np.arange(half) % n
    edge = np.round(np.cumsum([1] + [2] * (n - 1)) * half / (2 * n - 1)).astype(np.int64)
    return np.searchsorted(edge, np.arange(half), side="right")


def work(case):
    """Each input read once and each output written once; the multiplications and additions of the products."""
    e, d, n_kv = _ESIZE[case["dtype"]], case["d"], case["n_kv"]
    if case["op"] == "axes":
        T, heads = case["T"], case["n_q"]
        rows = min(T, case["max_pos"]) * case["rot"] * 4
        return {"bytes": 2 * T * (heads + 2 * n_kv) * d * e + (8 + 4 * case["axes"]) * T + rows + (2 * d * e if case["norm"] else 0),
                "flops": T * (heads + n_kv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if case["op"] == "weigh":
        heads = case["n_q"]
        see, drafts = _visible(case)
        _, lens = _lengths(case)
        pairs = int((drafts * (lens - drafts)).sum()) + int(see.sum())
        T, keys, new = int(drafts.sum()), int(lens[drafts > 0].sum()), int(drafts.sum())
        tables = 4 * int(np.ceil(lens / case["page"]).sum()) + 8 * case["S"] + (8 * T * ((case["n"] + 63) // 64) if case["mask"] == "tree" else 0)
        sums = 4 * keys * n_kv + (4 * (keys - new) * n_kv if case["decay"] else 0)
        return {"bytes": 2 * T * heads * d * e + 2 * keys * n_kv * d * e + sums + tables, "flops": 4 * pairs * heads * d}
    lens = _evicted_lengths(case)
    total = 12 * case["S"]
    for length in lens[lens > case["keep"]]:
        # the tokens before the first evicted one stay where they are: one part in (evicted + 1) of those that compete
        gone, compete = length - case["keep"], length - case["first"] - case["recent"]
        moved = max(0, case["keep"] - case["first"] - int(max(0, compete) / (gone + 1)))
        total += n_kv * (4 * length + 4 * case["keep"] + 2 * moved * (2 * d * e + 4)) + 4 * -(-length // case["page"])
    return {"bytes": int(total), "flops": 0}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _page_table(st, g, lens, page):
    """Pages of the requests, anywhere in the cache, with three to spare: the table (-1: none) and the page count."""
    used = -(-lens // page)
    n_pages, width = int(used.sum()) + 3, max(1, int(used.max()))
    ids = torch.randperm(n_pages, generator=g, device="cuda").int()
    at = torch.arange(width, device="cuda")[None, :]
    count = torch.from_numpy(used).cuda()[:, None]
    first = torch.cumsum(count, 0) - count
    st["table"] = torch.where(at < count, ids[(first + at).clamp(max=n_pages - 1)], torch.tensor(-1, device="cuda", dtype=torch.int32)).contiguous()
    st["width"], st["lens"], st["longest"] = width, torch.from_numpy(lens.astype(np.int32)).cuda(), int(lens.max())
    return n_pages


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt).mul_(scale)

    st = dict(case)
    n_kv, d, page = case["n_kv"], case["d"], case["page"]
    if case["op"] == "axes":
        T, n_q, width = case["T"], case["n_q"], (case["n_q"] + 2 * n_kv) * d
        if case["fused"]:       # one projection made q, k and v: rows of one matrix
            qkv = normal(T, width)
            st["q"], st["k"], st["v"] = qkv[:, : n_q * d], qkv[:, n_q * d: (n_q + n_kv) * d], qkv[:, (n_q + n_kv) * d:]
        else:
            st["q"], st["k"], st["v"] = normal(T, n_q * d), normal(T, n_kv * d), normal(T, n_kv * d)
        st["q_norm"] = (1 + normal(d, scale=0.1)) if case["norm"] else None
        st["k_norm"] = (1 + normal(d, scale=0.1)) if case["norm"] else None
        # the rotation's table as a server keeps it: cosines, then sines, of position * 10000^(-2i / rot)
        half = case["rot"] // 2
        angle = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * \
            torch.pow(10000.0, -torch.arange(half, device="cuda", dtype=torch.float64) / half)[None, :]
        st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        # patches of images and video frames, row by row, from some position on; every fifth run is text, whose axes agree
        run = torch.arange(T, device="cuda") // 64
        begin = torch.randint(0, max(1, case["max_pos"] - 16), (T // 64 + 1,), generator=g, device="cuda")[run]
        i = torch.arange(T, device="cuda") % 64
        patch = torch.stack([torch.zeros_like(i), i // 8, i % 8, i % 3], 1)[:, : case["axes"]]
        text = (run % 5 == 4)[:, None]
        st["positions"] = (begin[:, None] + torch.where(text, (i % 16)[:, None], patch)).clamp(max=case["max_pos"] - 1).int().contiguous()
        axis = _pair_axes(case)
        st["pair_axis"], st["axis"] = axis.astype(np.uint8).tobytes(), torch.from_numpy(axis).cuda()
        # every token gets a cache slot of its own, anywhere in the cache; one in 16 is padding and is not stored
        n_pages = (2 * T + page - 1) // page
        slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:T]
        slots[15::16] = -1
        st["slots"] = slots
        st["q_out"] = torch.empty(T, n_q * d, device="cuda", dtype=dt)
        st["eps"] = 1e-6
    elif case["op"] == "weigh":
        see, drafts = _visible(case)
        _, lens = _lengths(case)
        T, words = int(drafts.sum()), (case["n"] + 63) // 64
        n_pages = _page_table(st, g, lens, page)
        st["T"], st["words"], st["bits"] = T, words, None
        st["starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)).cuda()
        if case["mask"] == "tree":
            wide = np.zeros((T, words * 64), bool)
            wide[:, : case["n"]] = see
            packed = np.packbits(wide, axis=1, bitorder="little").view("<i8")
            st["bits"] = torch.from_numpy(np.ascontiguousarray(packed)).cuda()
        st["q"] = normal(T, case["n_q"] * d)
        st["scale"] = 1.0 / math.sqrt(d)
        st["out"] = torch.empty(T, case["n_q"] * d, device="cuda", dtype=dt)
        # what a few steps like this one left: a few tokens have most of the weight
        st["weights"] = torch.exp(2 * torch.randn(n_pages, n_kv, page, generator=g, device="cuda")) * (case["n_q"] // n_kv * case["n"] / case["max_len"])
    else:
        lens = _evicted_lengths(case)
        n_pages = _page_table(st, g, lens, page)
        scores = torch.exp(2 * torch.randn(n_pages, n_kv, page, generator=g, device="cuda"))
        st["scores"] = torch.round(scores * 8) / 8 if case["ties"] else scores
        st["weights"] = torch.exp(2 * torch.randn(n_pages, n_kv, page, generator=g, device="cuda"))
        st["budget"] = torch.full((case["S"],), case["keep"], dtype=torch.int32, device="cuda")
        st["kept"] = torch.zeros(case["S"], n_kv, case["keep"], dtype=torch.int32, device="cuda")
        st["new_lens"] = torch.zeros(case["S"], dtype=torch.int32, device="cuda")
    # the cache as earlier steps left it
    st["k_pages"], st["v_pages"] = normal(n_pages, n_kv, page, d), normal(n_pages, n_kv, page, d)
    if own:
        from segmented_gathered_rank_gb300 import lora
        st["lora"] = lora
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        st["kv"] = lora.KvPages(lora.LORA_BF16 if case["dtype"] == BF16 else lora.LORA_F32, st["k_pages"], st["v_pages"], n_pages,
                                page, n_kv, d, status=st["status"])
        if case["op"] == "weigh":
            size = lora.lora_tree_attention_weights_workspace_size(st["kv"], case["n_q"], case["S"], st["T"], st["width"])
            st["workspace"] = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    return st


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def run(st):
    return {"axes": _run_axes, "weigh": _run_weigh, "evict": _run_evict}[st["op"]](st)


def _run_axes(st):
    if own:
        st["lora"].lora_kv_append_axes(st["kv"], st["q"], st["k"], st["v"], st["T"], st["n_q"], st["positions"], st["axes"],
                                       st["pair_axis"], st["slots"], st["cos_sin"], st["max_pos"], st["rot"], st["interleaved"],
                                       st["q_out"], q_norm=st["q_norm"], k_norm=st["k_norm"], eps=st["eps"])
        return {"q": st["q_out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    T, d, dt, half = st["T"], st["d"], st["q"].dtype, st["rot"] // 2
    at = st["positions"].long()[:, st["axis"]]                       # [T, half] table rows
    pair = torch.arange(half, device=at.device)[None, :]
    cos, sin = st["cos_sin"][at, pair][:, None, :], st["cos_sin"][at, half + pair][:, None, :]

    def turned(x, weight):
        x = x.float().reshape(T, -1, d)
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + st["eps"]) * weight.float()
        a, b = (x[..., : 2 * half: 2], x[..., 1: 2 * half: 2]) if st["interleaved"] else (x[..., :half], x[..., half: 2 * half])
        y = [a * cos - b * sin, a * sin + b * cos]
        y = torch.stack(y, -1).flatten(-2) if st["interleaved"] else torch.cat(y, -1)
        return torch.cat([y, x[..., 2 * half:]], -1).to(dt)

    q, k = turned(st["q"], st["q_norm"]), turned(st["k"], st["k_norm"])
    keep = st["slots"] >= 0
    page, off = st["slots"][keep] // st["page"], st["slots"][keep] % st["page"]
    st["k_pages"][page, :, off] = k[keep]
    st["v_pages"][page, :, off] = st["v"].reshape(T, -1, d)[keep]
    return {"q": q.view(T, -1), "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _run_weigh(st):
    if own:
        st["lora"].lora_tree_attention_weights(st["kv"], st["weights"], st["decay"], st["q"], st["n_q"], st["starts"], st["S"], st["T"],
                                               st["lens"], st["table"], st["width"], st["bits"], st["words"], st["scale"], st["out"],
                                               st["workspace"])
        return {"out": st["out"], "weights": st["weights"]}
    S, T, n, n_kv, d, L = st["S"], st["T"], st["n"], st["n_kv"], st["d"], st["longest"]
    dev = st["q"].device
    at, i = torch.arange(L, device=dev), torch.arange(n, device=dev)
    starts, lens = st["starts"].long(), st["lens"].long()
    count = starts[1:] - starts[:-1]
    row = (starts[:-1, None] + i).clamp(max=T - 1)                               # [S, n] rows of q, padded
    page = st["table"][:, at // st["page"]].long().clamp(min=0)                  # [S, L]
    k = st["k_pages"][page, :, at % st["page"]].float().transpose(1, 2)          # [S, n_kv, L, d]
    v = st["v_pages"][page, :, at % st["page"]].float().transpose(1, 2)
    q = st["q"].float().view(T, n_kv, -1, d)[row].permute(0, 2, 3, 1, 4)         # [S, n_kv, g, n, d]
    s = (q.reshape(S, n_kv, -1, d) @ k.transpose(2, 3)).view(S, n_kv, -1, n, L) * st["scale"]
    j = at[None, :] - (lens - count)[:, None]                                    # [S, L] drafted index of a cached token
    if st["bits"] is None:
        see = (j[:, None, :] <= i[None, :, None])
    else:
        j0 = j.clamp(0, st["words"] * 64 - 1)
        word = torch.gather(st["bits"][row], 2, (j0 // 64)[:, None, :].expand(S, n, L))
        see = ((word >> (j0 % 64)[:, None, :]) & 1).bool() | (j[:, None, :] < 0)
    live = i[None, :] < count[:, None]
    see = (see & (at[None, :] < lens[:, None])[:, None, :] & live[:, :, None])[:, None, None]
    s = s.masked_fill_(~see, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    p = p / total.masked_fill(total == 0, 1.0)
    o = (p.view(S, n_kv, -1, L) @ v).view(S, n_kv, -1, n, d)
    o = o.permute(0, 3, 1, 2, 4).reshape(S * n, -1)[live.reshape(-1)].to(st["q"].dtype)
    gained = p.sum((2, 3)).transpose(1, 2)                                       # [S, L, n_kv]
    old = st["weights"][page, :, at % st["page"]]
    new = gained + torch.where((j < 0)[:, :, None], st["decay"] * old, 0.0)
    told = (at[None, :] < lens[:, None]) & (count > 0)[:, None]                  # requests with new tokens, their own tokens
    st["weights"][page[told], :, (at % st["page"]).expand(S, L)[told]] = new[told]
    return {"out": o, "weights": st["weights"]}


def _run_evict(st):
    if own:
        st["lora"].lora_kv_evict(st["kv"], st["scores"], st["weights"], st["S"], st["lens"], st["table"], st["width"], st["budget"],
                                 st["first"], st["recent"], st["kept"], st["keep"], st["new_lens"])
    else:
        keep, page, L = st["keep"], st["page"], st["longest"]
        dev = st["lens"].device
        lens = st["lens"].long()
        some = torch.nonzero(lens > keep)[:, 0]                                  # the requests that lose tokens
        if len(some):
            at = torch.arange(L, device=dev)
            pages = st["table"][some][:, at // page].long().clamp(min=0)         # [R, L]
            score = st["scores"][pages, :, at % page].transpose(1, 2)            # [R, n_kv, L]
            recent = min(st["recent"], keep)
            first = min(st["first"], keep - recent)
            length = lens[some][:, None, None]
            score = score.masked_fill((at < first) | (at >= length - recent), math.inf).masked_fill(at >= length, -math.inf)
            order = torch.sort(score, dim=2, descending=True, stable=True).indices[:, :, :keep]
            src = torch.sort(order, dim=2).values                                # [R, n_kv, keep]
            head = torch.arange(st["n_kv"], device=dev)[None, :, None]
            r = torch.arange(len(some), device=dev)[:, None, None]
            to = torch.arange(keep, device=dev).expand_as(src)
            for plane in (st["k_pages"], st["v_pages"], st["weights"]):
                plane[pages[r, to], head, to % page] = plane[pages[r, src], head, src % page]
            st["kept"][some] = src.int()
        st["new_lens"].copy_(lens.clamp(max=keep))
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"], "weights": st["weights"], "kept": st["kept"], "new_lens": st["new_lens"]}


# ----------------------------------------------------------------------------
# The definitions in 64 bits, request by request and head by head
# ----------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    return {"axes": _exact_axes, "weigh": _exact_weigh, "evict": _exact_evict}[case["op"]](st)


def _exact_axes(st):
    f64, d, half = torch.float64, st["d"], st["rot"] // 2
    turn = torch.empty(st["T"], half, dtype=torch.complex128, device="cuda")
    for pair, axis in enumerate(_pair_axes(st).tolist()):
        rows = st["cos_sin"][st["positions"][:, axis].long()].to(f64)
        turn[:, pair] = torch.complex(rows[:, pair], rows[:, half + pair])

    def head(x, weight):
        x = x.to(f64)
        x = x / torch.sqrt((x * x).sum(1) / d + st["eps"])[:, None] * weight.to(f64) if weight is not None else x.clone()
        first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if st["interleaved"] else (slice(0, half), slice(half, 2 * half))
        z = torch.complex(x[:, first], x[:, second]) * turn     # a rotation is a complex product
        x[:, first], x[:, second] = z.real, z.imag
        return x

    q = torch.cat([head(st["q"][:, h * d: (h + 1) * d], st["q_norm"]) for h in range(st["n_q"])], 1)
    k_pages, v_pages = st["k_pages"].to(f64), st["v_pages"].to(f64)
    at = st["slots"][st["slots"] >= 0]
    for h in range(st["n_kv"]):
        for pages, x in ((k_pages, head(st["k"][:, h * d: (h + 1) * d], st["k_norm"])), (v_pages, st["v"][:, h * d: (h + 1) * d].to(f64))):
            rows = pages[:, h].reshape(-1, d).clone()
            rows[at] = x[st["slots"] >= 0]
            pages[:, h] = rows.view(-1, st["page"], d)
    return {"q": q, "k_pages": k_pages, "v_pages": v_pages}


def _exact_weigh(st):
    f64, d, page, group = torch.float64, st["d"], st["page"], st["n_q"] // st["n_kv"]
    see, drafts = _visible(st)
    _, lens = _lengths(st)
    see = torch.from_numpy(see).cuda()
    out = torch.zeros(st["T"], st["n_q"], d, dtype=f64, device="cuda")
    weights = st["weights"].to(f64)
    begin = 0
    for s in range(st["S"]):
        n, length = int(drafts[s]), int(lens[s])
        end = begin + n
        if n and length:
            ids = st["table"][s, : -(-length // page)].long()
            mine = torch.cat([torch.ones(n, length - n, dtype=torch.bool, device="cuda"), see[begin:end, :n]], 1)
            some = mine.any(1)
            for h in range(st["n_kv"]):
                k = st["k_pages"][ids, h].reshape(-1, d)[:length].to(f64)
                v = st["v_pages"][ids, h].reshape(-1, d)[:length].to(f64)
                flat = weights[ids, h].reshape(-1)
                total = flat[:length] * st["decay"]
                total[length - n:] = 0
                for q_head in range(h * group, (h + 1) * group):
                    q = st["q"][begin:end, q_head * d: (q_head + 1) * d].to(f64)
                    p = torch.softmax((q @ k.t() * st["scale"]).masked_fill(~mine, -math.inf), 1)
                    out[begin:end, q_head][some] = (p @ v)[some]
                    total += p[some].sum(0)
                flat[:length] = total
                weights[ids, h] = flat.view(-1, page)
        begin = end
    return {"out": out.view(st["T"], -1), "weights": weights}


def _exact_evict(st):
    keep, page = st["keep"], st["page"]
    scores, lens, table = st["scores"].cpu().numpy(), st["lens"].tolist(), st["table"].cpu().numpy()
    planes = [st[name].to(torch.float64) for name in ("k_pages", "v_pages", "weights")]
    kept = np.zeros((st["S"], st["n_kv"], keep), np.int32)
    new_lens = np.minimum(lens, keep).astype(np.int32)
    recent = min(st["recent"], keep)
    first = min(st["first"], keep - recent)
    for s, length in enumerate(lens):
        if length <= keep:
            continue
        ids = table[s, : -(-length // page)].astype(np.int64)
        for h in range(st["n_kv"]):
            score = scores[ids, h].reshape(-1)[:length].astype(np.float64)
            middle = np.arange(first, length - recent)
            best = middle[np.lexsort((middle, -score[middle]))][: keep - first - recent]
            chosen = np.sort(np.concatenate([np.arange(first), best, np.arange(length - recent, length)]))
            kept[s, h] = chosen
            source, mine = torch.from_numpy(chosen).cuda(), torch.from_numpy(ids).cuda()
            for plane in planes:
                rows = plane[mine, h].reshape(len(ids) * page, -1)
                rows[:keep] = rows[source]
                plane[mine, h] = rows.view(plane[mine, h].shape)
    return {"k_pages": planes[0], "v_pages": planes[1], "weights": planes[2], "kept": torch.from_numpy(kept).cuda(),
            "new_lens": torch.from_numpy(new_lens).cuda()}
