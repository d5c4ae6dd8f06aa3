"""Cases, plain forms and exact results of the decode-step operators.

The operators are those of one attention block of a decode step under many
adapters: the base product of a projection from 4-bit weights
(``lora_w4_matvec``), the norm and rotation of queries and keys with the
append of keys and values to the paged cache (``lora_kv_append``), and the
attention of drafted tokens over that cache (``lora_tree_attention``).

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
        # One request decodes: the k projection (4096 -> 1024), symmetric codes.
        dict(name="w4_1", op="w4", dtype=BF16, T=1, h_in=4096, h_out=1024, group=128, zeros=False),
        # Five drafted tokens of one request, fp32 activations, sizes off every tile, small groups.
        dict(name="w4_odd_f32", op="w4", dtype=F32, T=5, h_in=4128, h_out=4001, group=32, zeros=True),
        # A tree of 64 drafted tokens through a wide projection.
        dict(name="w4_64", op="w4", dtype=BF16, T=64, h_in=4096, h_out=16384, group=128, zeros=True),
        # One request's new token: the smallest append.
        dict(name="append_1", op="append", dtype=BF16, T=1, n_q=32, n_kv=8, d=128, rot=128, page=16,
             interleaved=False, norm=True, fused=True, max_pos=8192),
        # A decode batch of 256 requests, one new token each.
        dict(name="append_256", op="append", dtype=BF16, T=256, n_q=32, n_kv=8, d=128, rot=128, page=16,
             interleaved=False, norm=True, fused=False, max_pos=32768),
        # A prefill batch: 8192 tokens, rotation of neighbouring pairs, no norms, one fused qkv matrix.
        dict(name="append_8192", op="append", dtype=BF16, T=8192, n_q=32, n_kv=8, d=128, rot=128, page=64,
             interleaved=True, norm=False, fused=True, max_pos=8192),
        # Odd everything: head width 80 with 20 rotated, 7 query heads on one kv head, fp32.
        dict(name="append_odd_f32", op="append", dtype=F32, T=333, n_q=7, n_kv=1, d=80, rot=20, page=8,
             interleaved=False, norm=True, fused=False, max_pos=2048),
        # One request decodes one token over a short context: the smallest attention.
        dict(name="attn_1", op="attn", dtype=BF16, S=1, n=1, max_len=777, n_q=32, n_kv=8, d=128, page=16,
             mask="chain", padded=False),
        # A decode batch: 128 requests of very different lengths, one token each.
        dict(name="attn_decode_128", op="attn", dtype=BF16, S=128, n=1, max_len=8192, n_q=32, n_kv=8, d=128, page=16,
             mask="chain", padded=False),
        # Eight requests verify trees of up to 64 drafted tokens over long contexts.
        dict(name="attn_tree_64", op="attn", dtype=BF16, S=8, n=64, max_len=16384, n_q=32, n_kv=8, d=128, page=64,
             mask="tree", padded=False),
        # Two requests verify small trees over very long contexts.
        dict(name="attn_long_16", op="attn", dtype=BF16, S=2, n=16, max_len=131072, n_q=32, n_kv=8, d=128, page=16,
             mask="tree", padded=False),
        # fp32, an odd head width, five requests with padded trees, some of them without any context.
        dict(name="attn_odd_f32", op="attn", dtype=F32, S=5, n=7, max_len=300, n_q=6, n_kv=2, d=80, page=8,
             mask="tree", padded=True),
    ]


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _spread(rng, lo, hi, unit=1):
    """A whole number of [lo, hi], spread over its logarithm; times `unit` it is off the grid of 1024 that listed cases lie on."""
    v = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return v - 1 if v * unit % 1024 == 0 else v


def draw(rng):
    """One more case: T, lengths and widths over their logarithm; costs at most the largest listed case of its operator."""
    op = rng.choice(["w4", "append", "attn"])
    cap = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        dtype = rng.choice([BF16, BF16, BF16, F32])
        if op == "w4":
            group = rng.choice([32, 64, 128])
            case = dict(op=op, dtype=dtype, T=_spread(rng, 1, 64), h_in=group * _spread(rng, 512 // group, 16384 // group, group),
                        h_out=_spread(rng, 256, 16384), group=group, zeros=rng.random() < 0.5)
        else:
            n_kv = rng.choice([1, 2, 4, 8])
            heads = dict(n_q=n_kv * rng.choice([1, 2, 4, 7, 8]), n_kv=n_kv, d=rng.choice([64, 80, 112, 128, 128, 256]),
                         page=rng.choice([1, 8, 16, 32, 64, 128]))
            if op == "append":
                rot = heads["d"] if rng.random() < 0.6 else 2 * rng.randint(1, heads["d"] // 2)
                case = dict(op=op, dtype=dtype, T=_spread(rng, 1, 8192), rot=rot, interleaved=rng.random() < 0.4,
                            norm=rng.random() < 0.6, fused=rng.random() < 0.5, max_pos=_spread(rng, 512, 131072), **heads)
                if case["fused"] and (case["n_q"] + 2 * n_kv) * case["d"] % 1024 == 0:
                    case["fused"] = False
            else:
                n = rng.choice([1, _spread(rng, 1, 128)])
                case = dict(op=op, dtype=dtype, S=_spread(rng, 1, 128), n=n, max_len=max(n, _spread(rng, 16, 131072)),
                            mask=rng.choice(["tree", "tree", "chain"]) if n > 1 else "chain",
                            padded=n > 1 and rng.random() < 0.4, **heads)
                plain = case["S"] * case["n_q"] * n * case["max_len"] + case["S"] * case["max_len"] * n_kv * heads["d"]
                if plain > 2 ** 31:     # the plain form pads every request to the longest one
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
    last quarter of a request's tokens are padding that sees no drafted token."""
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


def work(case):
    """Each input read once and each output written once; the multiplications and additions of the products."""
    e = _ESIZE[case["dtype"]]
    if case["op"] == "w4":
        T, hi, ho, groups = case["T"], case["h_in"], case["h_out"], case["h_in"] // case["group"]
        return {"bytes": ho * hi // 2 + ho * groups * (3 if case["zeros"] else 2) + e * T * (hi + ho), "flops": 2 * T * hi * ho}
    heads, d = case["n_q"], case["d"]
    if case["op"] == "append":
        T = case["T"]
        rows = min(T, case["max_pos"]) * case["rot"] * 4
        return {"bytes": 2 * T * (heads + 2 * case["n_kv"]) * d * e + 12 * T + rows + (2 * d * e if case["norm"] else 0),
                "flops": T * (heads + case["n_kv"]) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    see, drafts = _visible(case)
    _, lens = _lengths(case)
    pairs = int((drafts * (lens - drafts)).sum()) + int(see.sum())
    T, keys = int(drafts.sum()), int(lens[drafts > 0].sum())
    tables = 4 * int(np.ceil(lens / case["page"]).sum()) + 8 * case["S"] + (8 * T * ((case["n"] + 63) // 64) if case["mask"] == "tree" else 0)
    return {"bytes": 2 * T * heads * d * e + 2 * keys * case["n_kv"] * d * e + tables, "flops": 4 * pairs * heads * d}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dt).mul_(scale)

    st = dict(case)
    if case["op"] == "w4":
        T, hi, ho, groups = case["T"], case["h_in"], case["h_out"], case["h_in"] // case["group"]
        st["x"] = normal(T, hi)
        st["codes"] = torch.randint(0, 256, (ho, hi // 2), generator=g, device="cuda", dtype=torch.uint8)
        st["scales"] = (torch.rand(ho, groups, generator=g, device="cuda") * 0.75 + 0.25).mul_(0.3 / math.sqrt(hi)).to(torch.bfloat16)
        st["zeros"] = torch.randint(4, 12, (ho, groups), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        st["y"] = torch.empty(T, ho, device="cuda", dtype=dt)
        if own:
            from segmented_gathered_rank_gb300 import lora
            st["lora"], st["code"] = lora, lora.LORA_BF16 if case["dtype"] == BF16 else lora.LORA_F32
        return st

    n_q, n_kv, d, page = case["n_q"], case["n_kv"], case["d"], case["page"]
    if case["op"] == "append":
        T, width = case["T"], (n_q + 2 * n_kv) * d
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
        st["positions"] = torch.randint(0, case["max_pos"], (T,), generator=g, device="cuda", dtype=torch.int32)
        # every token gets a cache slot of its own, anywhere in the cache; one in 16 is padding and is not stored
        n_pages = (2 * T + page - 1) // page
        slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:T]
        slots[15::16] = -1
        st["slots"] = slots
        # cache and rows written by earlier steps
        st["k_pages"], st["v_pages"] = normal(n_pages, n_kv, page, d), normal(n_pages, n_kv, page, d)
        st["q_out"] = torch.empty(T, n_q * d, device="cuda", dtype=dt)
        st["eps"] = 1e-6
    else:
        see, drafts = _visible(case)
        _, lens = _lengths(case)
        S, T, words = case["S"], int(drafts.sum()), (case["n"] + 63) // 64
        used = -(-lens // page)
        n_pages, width = int(used.sum()) + 3, int(used.max())
        ids = torch.randperm(n_pages, generator=g, device="cuda").int()
        at = torch.arange(width, device="cuda")[None, :]
        count = torch.from_numpy(used).cuda()[:, None]
        first = torch.cumsum(count, 0) - count
        st["table"] = torch.where(at < count, ids[(first + at).clamp(max=n_pages - 1)], torch.tensor(-1, device="cuda", dtype=torch.int32)).contiguous()
        st["width"], st["T"], st["words"], st["longest"] = width, T, words, int(lens.max())
        st["starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)).cuda()
        st["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        st["bits"] = None
        if case["mask"] == "tree":
            wide = np.zeros((T, words * 64), bool)
            wide[:, : case["n"]] = see
            packed = np.packbits(wide, axis=1, bitorder="little").view("<i8")
            st["bits"] = torch.from_numpy(np.ascontiguousarray(packed)).cuda()
        st["q"] = normal(T, n_q * d)
        st["k_pages"], st["v_pages"] = normal(n_pages, n_kv, page, d), normal(n_pages, n_kv, page, d)
        st["scale"] = 1.0 / math.sqrt(d)
        st["out"] = torch.empty(T, n_q * d, device="cuda", dtype=dt)
    if own:
        from segmented_gathered_rank_gb300 import lora
        st["lora"] = lora
        st["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        st["kv"] = lora.KvPages(lora.LORA_BF16 if case["dtype"] == BF16 else lora.LORA_F32, st["k_pages"], st["v_pages"], n_pages,
                                page, n_kv, d, status=st["status"])
        if case["op"] == "attn":
            size = lora.lora_tree_attention_workspace_size(st["kv"], n_q, case["S"], T)
            st["workspace"] = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    return st


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def run(st):
    return {"w4": _run_w4, "append": _run_append, "attn": _run_attn}[st["op"]](st)


def _run_w4(st):
    if own:
        st["lora"].lora_w4_matvec(st["code"], st["x"], st["T"], st["h_in"], st["codes"], st["scales"], st["zeros"], st["group"],
                                  st["h_out"], st["y"])
        return st["y"]
    c = st["codes"]
    w = torch.stack([c & 15, c >> 4], 2).reshape(st["h_out"], -1, st["group"]).float()
    w = w - (st["zeros"].float()[:, :, None] if st["zeros"] is not None else 8.0)
    w = (w * st["scales"].float()[:, :, None]).reshape(st["h_out"], st["h_in"])
    return (st["x"].float() @ w.t()).to(st["x"].dtype)


def _normed_and_turned(x, weight, eps, cos, sin, interleaved):
    """Heads [T, H, d] in fp32: x / rms(x) * weight, then the first 2 * cos.shape[-1] elements rotated."""
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.float()
    half = cos.shape[-1]
    a, b = (x[..., : 2 * half: 2], x[..., 1: 2 * half: 2]) if interleaved else (x[..., :half], x[..., half: 2 * half])
    c, s = cos[:, None, :], sin[:, None, :]
    turned = [a * c - b * s, a * s + b * c]
    turned = torch.stack(turned, -1).flatten(-2) if interleaved else torch.cat(turned, -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _run_append(st):
    if own:
        st["lora"].lora_kv_append(st["kv"], st["q"], st["k"], st["v"], st["T"], st["n_q"], st["positions"], st["slots"], st["cos_sin"],
                                  st["max_pos"], st["rot"], st["interleaved"], st["q_out"], q_norm=st["q_norm"], k_norm=st["k_norm"],
                                  eps=st["eps"])
        return {"q": st["q_out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    T, d, dt = st["T"], st["d"], st["q"].dtype
    rows = st["cos_sin"][st["positions"].long()]
    cos, sin = rows.chunk(2, -1)
    q = _normed_and_turned(st["q"].float().view(T, -1, d), st["q_norm"], st["eps"], cos, sin, st["interleaved"])
    k = _normed_and_turned(st["k"].float().view(T, -1, d), st["k_norm"], st["eps"], cos, sin, st["interleaved"])
    keep = st["slots"] >= 0
    page, at = st["slots"][keep] // st["page"], st["slots"][keep] % st["page"]
    st["k_pages"][page, :, at] = k.to(dt)[keep]
    st["v_pages"][page, :, at] = st["v"].reshape(T, -1, d)[keep]
    return {"q": q.to(dt).view(T, -1), "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _run_attn(st):
    if own:
        st["lora"].lora_tree_attention(st["kv"], st["q"], st["n_q"], st["starts"], st["S"], st["T"], st["lens"], st["table"], st["width"],
                                       st["bits"], st["words"], st["scale"], st["out"], st["workspace"])
        return st["out"]
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
    see = (see & (at[None, :] < lens[:, None])[:, None, :])[:, None, None]
    s = s.masked_fill_(~see, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1)[..., None]
    o = (p.view(S, n_kv, -1, L) @ v).view(S, n_kv, -1, n, d) / total.masked_fill(total == 0, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(S * n, -1)
    return o[(i[None, :] < count[:, None]).reshape(-1)].to(st["q"].dtype)


# ----------------------------------------------------------------------------
# The definitions in 64 bits, request by request and head by head
# ----------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "w4":
        y = torch.zeros(case["T"], case["h_out"], dtype=f64, device="cuda")
        x = st["x"].to(f64)
        for k in range(case["h_in"] // case["group"]):     # sum over groups of scale * (sum x * code - zero * sum x)
            part = x[:, k * case["group"]: (k + 1) * case["group"]]
            two = st["codes"][:, k * case["group"] // 2: (k + 1) * case["group"] // 2].to(f64)
            high = torch.floor(two / 16)
            inner = part[:, 0::2] @ (two - 16 * high).t() + part[:, 1::2] @ high.t()
            zero = st["zeros"][:, k].to(f64) if case["zeros"] else torch.full((case["h_out"],), 8.0, dtype=f64, device="cuda")
            y += st["scales"][:, k].to(f64) * (inner - part.sum(1)[:, None] * zero)
        return y
    d = case["d"]
    if case["op"] == "append":
        half = case["rot"] // 2
        table = st["cos_sin"].to(f64)[st["positions"].long()]
        turn = torch.complex(table[:, :half], table[:, half:])

        def head(x, weight):
            x = x.to(f64)
            if weight is not None:
                x = x / torch.sqrt((x * x).sum(1) / d + st["eps"])[:, None] * weight.to(f64)
            else:
                x = x.clone()
            first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (slice(0, half), slice(half, 2 * half))
            z = torch.complex(x[:, first], x[:, second]) * turn     # a rotation is a complex product
            x[:, first], x[:, second] = z.real, z.imag
            return x

        q = torch.cat([head(st["q"][:, h * d: (h + 1) * d], st["q_norm"]) for h in range(case["n_q"])], 1)
        k_pages, v_pages = st["k_pages"].to(f64), st["v_pages"].to(f64)
        at = st["slots"][st["slots"] >= 0]
        for h in range(case["n_kv"]):
            for pages, x in ((k_pages, head(st["k"][:, h * d: (h + 1) * d], st["k_norm"])), (v_pages, st["v"][:, h * d: (h + 1) * d].to(f64))):
                rows = pages[:, h].reshape(-1, d).clone()
                rows[at] = x[st["slots"] >= 0]
                pages[:, h] = rows.view(-1, case["page"], d)
        return {"q": q, "k_pages": k_pages, "v_pages": v_pages}
    see, drafts = _visible(case)
    _, lens = _lengths(case)
    see = torch.from_numpy(see).cuda()
    out = torch.zeros(st["T"], case["n_q"], d, dtype=f64, device="cuda")
    group, begin = case["n_q"] // case["n_kv"], 0
    for s in range(case["S"]):
        n, length = int(drafts[s]), int(lens[s])
        end = begin + n
        if n and length:
            ids = st["table"][s, : -(-length // case["page"])].long()
            mine = torch.cat([torch.ones(n, length - n, dtype=torch.bool, device="cuda"), see[begin:end, :n]], 1)
            some = mine.any(1)
            for h in range(case["n_kv"]):
                k = st["k_pages"][ids, h].reshape(-1, d)[:length].to(f64)
                v = st["v_pages"][ids, h].reshape(-1, d)[:length].to(f64)
                for q_head in range(h * group, (h + 1) * group):
                    q = st["q"][begin:end, q_head * d: (q_head + 1) * d].to(f64)
                    p = torch.softmax((q @ k.t() * st["scale"]).masked_fill(~mine, -math.inf), 1)
                    out[begin:end, q_head][some] = (p @ v)[some]
        begin = end
    return out.view(st["T"], -1)
