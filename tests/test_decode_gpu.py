"""Decode-step operators on the GPU against their float64 definitions (bounds: tests/decode_cases.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from oracle import decode as D  # noqa: E402
from segmented_gathered_rank_gb300 import inputs as I  # noqa: E402
from segmented_gathered_rank_gb300 import lora as L  # noqa: E402
from tests import decode_cases as C  # noqa: E402

CODE = {I.BF16: L.LORA_BF16, I.F32: L.LORA_F32}
TORCH = {I.BF16: torch.bfloat16, I.F32: torch.float32}


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def assert_within(got, ref, bound):
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - ref) / bound)), np.argwhere(bad)[:4].tolist())


# ----------------------------------------------------------------------------
# 4-bit weights
# ----------------------------------------------------------------------------
W4_CASES = [   # T, h_in, h_out, group, zeros
    (1, 128, 1, 128, False), (1, 4096, 1024, 128, False), (1, 32, 17, 32, True), (2, 64, 16, 64, True),
    (3, 1056, 1001, 32, True), (5, 4160, 130, 64, False), (7, 2176, 515, 128, True), (8, 512, 256, 32, False),
    (9, 640, 100, 128, True), (16, 4096, 48, 64, True), (17, 1024, 333, 32, True), (31, 768, 64, 64, False),
    (33, 896, 77, 128, True), (64, 2048, 200, 128, True), (65, 256, 40, 32, False), (130, 512, 129, 64, True),
    (1, 16384, 260, 32, True), (4, 14336, 300, 128, False), (64, 96, 1500, 32, True)]


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("case", W4_CASES, ids=lambda c: "-".join(map(str, c)))
def test_w4_matvec(case, dtype):
    T, h_in, h_out, group, zeros = case
    x, codes, scales, z = C.w4_case(sum(case[:4]), dtype, T, h_in, h_out, group, zeros)
    ref, mag = D.w4_matvec(x, codes, scales, z, group)
    y = torch.full((T, h_out), float("nan"), dtype=TORCH[dtype], device="cuda")
    L.lora_w4_matvec(CODE[dtype], C.device(x, dtype), T, h_in, cuda(codes), cuda(scales).to(torch.bfloat16), cuda(z), group,
                     h_out, y)
    assert_within(host(y), ref, C.w4_bound(ref, mag, h_in, group, dtype))


def test_w4_writes_only_its_rows_and_repeats_bit_for_bit():
    x, codes, scales, z = C.w4_case(5, I.BF16, 3, 512, 37, 64, True)
    args = (C.device(x, I.BF16), 3, 512, cuda(codes), cuda(scales).to(torch.bfloat16), cuda(z), 64, 37)
    y = torch.full((4, 37), 7.0, dtype=torch.bfloat16, device="cuda")
    L.lora_w4_matvec(L.LORA_BF16, *args, y)
    again = torch.full((4, 37), 7.0, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.lora_w4_matvec(L.LORA_BF16, *args, again)
    torch.cuda.synchronize()
    assert torch.equal(y, again) and bool((y[3] == 7).all())


def test_w4_nan_and_inf_activations_reach_their_own_rows_only():
    x, codes, scales, z = C.w4_case(6, I.BF16, 4, 256, 24, 64, False)
    codes[:] = 0x99
    x[1, 5], x[2, 200] = np.nan, np.inf
    for dtype in (I.BF16, I.F32):
        y = torch.empty((4, 24), dtype=TORCH[dtype], device="cuda")
        L.lora_w4_matvec(CODE[dtype], C.device(x, dtype), 4, 256, cuda(codes), cuda(scales).to(torch.bfloat16), None, 64, 24, y)
        y = host(y)
        assert np.isfinite(y[[0, 3]]).all() and np.isnan(y[1]).all() and np.isposinf(y[2]).all()


def test_w4_refusals():
    x = torch.zeros((2, 128), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((8, 64), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((8, 4), dtype=torch.bfloat16, device="cuda")
    y = torch.full((2, 8), 3.0, dtype=torch.bfloat16, device="cuda")

    def status(dtype=L.LORA_BF16, x=x, T=2, h_in=128, codes=codes, scales=scales, group=32, h_out=8, y=y):
        n = L.lora_launch_count()
        try:
            L.lora_w4_matvec(dtype, x, T, h_in, codes, scales, None, group, h_out, y)
        except L.LoraError as e:
            assert L.lora_launch_count() == n
            return e.status
        return 0

    assert status(T=0) == 0 and bool((y == 3).all())
    assert status(dtype=9) == L.LORA_ERR_ARG
    assert status(T=-1) == L.LORA_ERR_ARG
    assert status(x=None) == L.LORA_ERR_ARG
    assert status(y=None) == L.LORA_ERR_ARG
    assert status(h_out=0) == L.LORA_ERR_ARG
    assert status(group=16) == L.LORA_ERR_SHAPE
    assert status(group=96) == L.LORA_ERR_SHAPE
    assert status(h_in=144) == L.LORA_ERR_SHAPE
    assert status(codes=codes.view(-1)[1:]) == L.LORA_ERR_ARG      # misaligned


# ----------------------------------------------------------------------------
# Norm, rotation, append
# ----------------------------------------------------------------------------
APPEND_CASES = [   # T, n_q, n_kv, d, rot, page, interleaved, norm, fused
    (1, 32, 8, 128, 128, 16, False, True, True), (5, 4, 4, 64, 64, 1, True, False, True),
    (7, 7, 1, 80, 20, 8, False, True, False), (3, 2, 2, 8, 2, 4, False, True, False), (4, 2, 1, 8, 6, 4, True, True, True),
    (33, 16, 2, 256, 256, 64, False, True, True), (9, 6, 3, 112, 42, 32, False, True, True),
    (17, 8, 8, 96, 96, 128, False, False, False), (6, 0, 2, 128, 64, 16, False, True, False),
    (300, 28, 4, 128, 128, 16, True, True, True), (65, 40, 8, 192, 190, 1024, False, True, True),
    (2, 3, 1, 24, 0, 2, False, True, False), (1100, 8, 2, 64, 32, 16, False, False, True)]


def append_case(case, dtype, seed):
    T, n_q, n_kv, d, rot, page, interleaved, norm, fused = case
    rng = np.random.default_rng(seed)
    x = C.store(rng.normal(0, 2, (T, (n_q + 2 * n_kv) * d)), dtype)
    q, k, v = x[:, : n_q * d], x[:, n_q * d: (n_q + n_kv) * d], x[:, (n_q + n_kv) * d:]
    qn, kn = (C.store(rng.normal(1, 0.2, d), dtype) for _ in range(2)) if norm else (None, None)
    n_pos = 97
    angle = rng.uniform(-4, 4, (n_pos, rot // 2))
    cos_sin = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    positions = rng.integers(0, n_pos, T).astype(np.int32)
    n_pages = -(-2 * T // page) + 1
    slots = rng.permutation(n_pages * page)[:T].astype(np.int64)
    slots[3::7] = -1
    kp, vp = (C.store(rng.normal(0, 1, (n_pages, n_kv, page, d)), dtype) for _ in range(2))
    return q, k, v, qn, kn, cos_sin, positions, slots, kp, vp


def run_append(case, dtype, arrays, in_place=False, status=None, stream=None):
    T, n_q, n_kv, d, rot, page, interleaved, norm, fused = case
    q, k, v, qn, kn, cos_sin, positions, slots, kp, vp = arrays
    kd, vd = C.device(kp, dtype), C.device(vp, dtype)
    if fused:
        x = C.device(np.concatenate([q, k, v], 1), dtype)
        qd, k2, v2 = x[:, : n_q * d], x[:, n_q * d: (n_q + n_kv) * d], x[:, (n_q + n_kv) * d:]
    else:
        qd, k2, v2 = (C.device(a, dtype) for a in (q, k, v))
    out = qd if in_place else torch.full((T, n_q * d), float("nan"), dtype=TORCH[dtype], device="cuda")
    opt = lambda a: None if a is None else C.device(a, dtype)  # noqa: E731
    kv = L.KvPages(CODE[dtype], kd, vd, len(kp), page, n_kv, d, status=status)
    L.lora_kv_append(kv, qd if n_q else None, k2, v2, T, n_q, cuda(positions), cuda(slots), cuda(cos_sin) if rot else None,
                     len(cos_sin), rot, interleaved, out if n_q else None, q_norm=opt(qn), k_norm=opt(kn), eps=1e-5, stream=stream)
    torch.cuda.synchronize()
    return host(out).reshape(T, n_q, d), host(kd), host(vd)


def append_bound(ref, dtype, d):
    head = np.abs(ref).max(-1, keepdims=True) if ref.size else np.abs(ref)
    return (2.0 ** -8 if dtype == I.BF16 else 0.0) * np.abs(ref) + (2 * np.log2(d) + 24) * 2 * C.U * head * 2 ** 0.5 + 1e-30


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: "-".join(map(str, c)))
def test_kv_append(case, dtype):
    T, n_q, n_kv, d, rot, page, interleaved, norm, fused = case
    arrays = append_case(case, dtype, T + d)
    q, k, v, qn, kn, cos_sin, positions, slots, kp, vp = arrays
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_append(case, dtype, arrays, status=status)
    ref = D.append(q.reshape(T, n_q, d).astype(np.float64), k.reshape(T, n_kv, d).astype(np.float64), v.reshape(T, n_kv, d),
                   positions, slots, cos_sin, rot, interleaved, qn, kn, float(np.float32(1e-5)), kp, vp)
    assert int(status) == 0
    assert_within(got[0], ref[0], append_bound(ref[0], dtype, d))
    assert_within(got[1], ref[1], append_bound(ref[1], dtype, d))
    assert np.array_equal(got[2], ref[2])
    written = np.zeros((len(kp), page), bool)
    for s in slots[slots >= 0]:
        written[s // page, s % page] = True
    keep = ~written[:, None, :, None] & np.ones_like(kp, bool)
    assert np.array_equal(got[1][keep], kp.astype(np.float64)[keep])     # slots that no token names are untouched
    if not fused and n_q:                                                # queries rotated in place
        again = run_append(case, dtype, arrays, in_place=True)
        assert np.array_equal(again[0], got[0]) and np.array_equal(again[1], got[1])


def test_append_flags_bad_slots_and_positions():
    case = (4, 2, 1, 16, 8, 4, False, False, False)
    arrays = list(append_case(case, I.F32, 3))
    arrays[6] = np.array([0, -5, 97, 3], np.int32)
    arrays[7] = np.array([0, 1, 2, len(arrays[8]) * 4], np.int64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, kp, vp = run_append(case, I.F32, arrays, status=status)
    assert int(status) == L.LORA_DEV_BAD_SLOT | L.LORA_DEV_BAD_POSITION
    ok = np.array(arrays[6])
    ok[1], ok[2] = 0, 96                                  # positions are clamped into the table
    slots = np.array(arrays[7])
    slots[3] = -1
    ref = D.append(arrays[0].reshape(4, 2, 16), arrays[1].reshape(4, 1, 16), arrays[2].reshape(4, 1, 16), ok, slots, arrays[5], 8, False,
                   None, None, 0.0, arrays[8], arrays[9])
    assert_within(q, ref[0], append_bound(ref[0], I.F32, 16))
    assert_within(kp, ref[1], append_bound(ref[1], I.F32, 16))
    assert np.array_equal(vp, ref[2])
    run_append(case, I.F32, arrays)                       # without a status word


def test_append_slots_beyond_32_bits_of_elements():
    n_pages, page, d = 140000, 128, 128                  # 2.3e9 elements a side
    kd = torch.zeros((n_pages, 1, page, d), dtype=torch.bfloat16, device="cuda")
    vd = torch.zeros_like(kd)
    kv = L.KvPages(L.LORA_BF16, kd, vd, n_pages, page, 1, d)
    k = torch.randn(2, d, device="cuda").bfloat16()
    v = torch.randn(2, d, device="cuda").bfloat16()
    slots = torch.tensor([n_pages * page - 1, 17000000], device="cuda")
    L.lora_kv_append(kv, None, k, v, 2, 0, None, slots, None, 0, 0, False, None)
    rows_k, rows_v = kd.view(-1, d), vd.view(-1, d)
    assert torch.equal(rows_k[slots], k) and torch.equal(rows_v[slots], v)
    assert int((rows_k != 0).any(1).sum()) == 2
    # attention over the far pages
    q = torch.zeros(2, d, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[n_pages - 1], [17000000 // page]], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    lens = torch.tensor([page, page], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(L.lora_tree_attention_workspace_size(kv, 1, 2, 2), dtype=torch.uint8, device="cuda")
    L.lora_tree_attention(kv, q, 1, starts, 2, 2, lens, table, 1, None, 0, 1.0, out, ws)
    ref = torch.stack([v[0].float() / page, v[1].float() / page])
    assert torch.allclose(out.float(), ref, rtol=2.0 ** -7, atol=0)


def test_append_refusals():
    kd = torch.zeros((4, 2, 8, 16), dtype=torch.bfloat16, device="cuda")
    vd = torch.zeros_like(kd)
    q, k = torch.zeros((3, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, 32), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    cs = torch.zeros((5, 16), device="cuda")

    def status(dtype=L.LORA_BF16, page=8, n_kv=2, d=16, n_pages=4, q=q, k=k, T=3, n_q=4, pos=pos, slots=slots, cs=cs, n_pos=5,
               rot=16, q_out=q, eps=1e-6):
        kv = L.KvPages(dtype, kd, vd, 4, 8, 2, 16)
        kv.page_size, kv.n_kv_heads, kv.head_dim, kv.n_pages = page, n_kv, d, n_pages
        n = L.lora_launch_count()
        try:
            L.lora_kv_append(kv, q, k, k, T, n_q, pos, slots, cs, n_pos, rot, False, q_out, eps=eps)
        except L.LoraError as e:
            assert L.lora_launch_count() == n
            return e.status
        return 0

    assert status(T=0) == 0
    assert status(dtype=5) == L.LORA_ERR_ARG
    assert status(page=12) == L.LORA_ERR_SHAPE
    assert status(page=2048) == L.LORA_ERR_SHAPE
    assert status(d=12) == L.LORA_ERR_SHAPE
    assert status(d=264) == L.LORA_ERR_SHAPE
    assert status(n_q=5) == L.LORA_ERR_SHAPE
    assert status(rot=5) == L.LORA_ERR_SHAPE
    assert status(rot=18) == L.LORA_ERR_SHAPE
    assert status(n_kv=4) == L.LORA_ERR_SHAPE            # k rows too short for 4 heads
    assert status(n_pages=0) == L.LORA_ERR_ARG
    assert status(T=-1) == L.LORA_ERR_ARG
    assert status(pos=None) == L.LORA_ERR_ARG
    assert status(slots=None) == L.LORA_ERR_ARG
    assert status(cs=None) == L.LORA_ERR_ARG
    assert status(n_pos=0) == L.LORA_ERR_ARG
    assert status(q_out=None) == L.LORA_ERR_ARG
    assert status(eps=-1.0) == L.LORA_ERR_ARG


# ----------------------------------------------------------------------------
# Attention
# ----------------------------------------------------------------------------
def run_attention(c, status=None, poison=0, out=None, k=None, v=None, table=None, lens=None, starts=None):
    kd, vd = C.device(c.k if k is None else k, c.dtype), C.device(c.v if v is None else v, c.dtype)
    kv = L.KvPages(CODE[c.dtype], kd, vd, c.n_pages, c.page, c.n_kv, c.d, status=status)
    q = C.device(c.q, c.dtype)
    o = q if out == "q" else torch.full_like(q, float("nan"))
    size = L.lora_tree_attention_workspace_size(kv, c.n_q, c.S, c.T)
    ws = torch.full((max(16, size),), poison, dtype=torch.uint8, device="cuda")
    L.lora_tree_attention(kv, q, c.n_q, cuda(c.starts if starts is None else starts), c.S, c.T, cuda(c.lens if lens is None else lens),
                          cuda(c.table if table is None else table), c.max_pages, cuda(c.bits), c.words, c.scale, o, ws)
    torch.cuda.synchronize()
    return o.float().cpu().numpy().astype(np.float64)


def check_attention(c):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_attention(c, status)
    ref, mag, big = D.tree_attention(c.q, c.k, c.v, c.starts, c.lens, c.table, c.masks, c.scale)
    assert int(status) == 0
    assert_within(got, ref, c.bound(ref, mag, big))
    assert np.array_equal(run_attention(c, poison=255), got)       # bit for bit, whatever the workspace held
    return got


ATTN_CASES = [   # requests, n_q, n_kv, d, page, mask
    ([(1, 1)], 4, 4, 128, 16, None),
    ([(1, 777)], 32, 8, 128, 16, None),
    ([(1, 64), (1, 65), (1, 63), (1, 128), (1, 1), (1, 129)], 8, 2, 128, 16, None),
    ([(1, 300), (1, 17), (1, 0 + 1), (1, 2000)], 8, 8, 64, 1, None),
    ([(7, 90), (3, 3), (0, 40), (5, 6), (0, 0), (7, 200)], 6, 2, 80, 8, "tree"),
    ([(16, 1000), (9, 500), (16, 16)], 32, 8, 128, 16, "tree"),
    ([(64, 700), (33, 4000), (50, 50)], 32, 8, 128, 64, "tree"),
    ([(64, 64), (64, 65), (63, 127), (1, 256), (64, 1000)], 16, 4, 64, 32, "random"),
    ([(65, 300), (128, 1024), (100, 101)], 8, 2, 128, 128, "tree"),
    ([(100, 2500), (17, 400)], 14, 2, 112, 16, "random"),
    ([(300, 300), (129, 777), (1, 50)], 8, 2, 128, 16, None),
    ([(200, 1500), (40, 40)], 16, 2, 64, 8, None),
    ([(2, 333), (6, 1000)], 8, 1, 256, 16, "tree"),
    ([(40, 700), (20, 90)], 8, 2, 256, 64, "tree"),
    ([(3, 70)], 5, 1, 8, 2, "tree"),
    ([(12, 150), (4, 1030)], 12, 4, 192, 1024, "tree"),
    ([(1, 20000)], 8, 2, 128, 16, None),
    ([(16, 20011)], 8, 2, 128, 64, "tree"),
    ([(64, 9001), (64, 70)], 8, 2, 128, 16, "tree"),
    ([(1, 37 * (i % 9) + 1) for i in range(70)], 14, 2, 128, 16, None),
    ([(i % 5, 11 * (i % 13) + i % 5) for i in range(600)], 2, 1, 64, 16, "tree")]


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("case", range(len(ATTN_CASES)))
def test_tree_attention(case, dtype):
    requests, n_q, n_kv, d, page, mask = ATTN_CASES[case]
    check_attention(C.Attention(100 + case, dtype, requests, n_q, n_kv, d, page, mask=mask))


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("heads", [(4, 4), (16, 2), (128, 1)])
def test_attention_rows_that_see_nothing(dtype, heads):
    def half_empty(rng, n):
        m = C.tree_masks(rng, n, "tree")
        m[n // 2:] = False
        return m
    c = C.Attention(7, dtype, [(12, 12), (4, 30), (1, 1)], *heads, 64, 16, mask=half_empty)
    got = check_attention(c)
    assert not got[6:12].any() and not got[16].any() and got[:6].all() and got[12:16].all()


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (32, 2)])
def test_attention_non_finite_drafts_reach_only_their_descendants(dtype, bad, heads):
    c = C.Attention(8, dtype, [(20, 83), (9, 9), (8, 40)], *heads, 64, 16, mask="tree")
    clean = run_attention(c)
    k, v = c.k.copy(), c.v.copy()
    j = 3
    for s in range(3):                                   # drafted token 3 of every request holds bad values
        at = int(c.lens[s]) - (int(c.starts[s + 1]) - int(c.starts[s])) + j
        page, off = c.table[s, at // 16], at % 16
        v[page, :, off] = bad
        if s:
            k[page, :, off] = bad
    got = run_attention(c, k=k, v=v)
    see = np.concatenate([m[:, j] for m in c.masks])
    assert np.array_equal(got[~see], clean[~see])
    assert see.any() and not np.isfinite(got[:20][see[:20]]).any()


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
def test_attention_large_scores_and_long_ties(dtype):
    # scores far apart (one key takes all) and equal keys (every probability the same)
    c = C.Attention(9, dtype, [(2, 600), (24, 260)], 8, 2, 64, 16, mask="tree", scale=30.0)
    check_attention(c)
    c = C.Attention(10, dtype, [(3, 5000)], 4, 1, 128, 16, mask="tree")
    c.q[...] = 0
    check_attention(c)


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("case", [4, 6, 16])
def test_attention_out_may_be_q(dtype, case):
    requests, n_q, n_kv, d, page, mask = ATTN_CASES[case]
    c = C.Attention(100 + case, dtype, requests, n_q, n_kv, d, page, mask=mask)
    assert np.array_equal(run_attention(c, out="q"), run_attention(c))


def test_attention_drafts_beyond_the_mask_words_are_not_visible():
    c = C.Attention(11, I.BF16, [(80, 100)], 4, 2, 64, 16, mask="tree", words=1)
    c.masks[0][:, 64:] = False
    check_attention(c)


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("n", [2, 40])
def test_attention_flags_bad_tables(dtype, n):
    c = C.Attention(12, dtype, [(n, 90), (n, 70), (n, 200)], 8, 2, 64, 16, mask="tree", garbage=0.0)
    good = run_attention(c)
    ref, mag, big = D.tree_attention(c.q, c.k, c.v, c.starts, c.lens, c.table, c.masks, c.scale)
    bound = c.bound(ref, mag, big)

    def flagged(**kw):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run_attention(c, status, **kw)
        run_attention(c, None, **kw)                     # without a status word
        return int(status), got

    table = c.table.copy()
    table[1, 2], table[1, 3] = c.n_pages, -3
    word, got = flagged(table=table)
    assert word == L.LORA_DEV_BAD_PAGE
    keep = np.r_[0:n, 2 * n: 3 * n]
    assert np.array_equal(got[keep], good[keep])
    for bad in (n - 1, -4, 16 * c.max_pages + 1):
        lens = c.lens.copy()
        lens[1] = bad
        word, got = flagged(lens=lens)
        assert word & L.LORA_DEV_BAD_LENGTH and word & ~(L.LORA_DEV_BAD_LENGTH | L.LORA_DEV_BAD_PAGE) == 0
        assert_within(got[keep], ref[keep], bound[keep])       # (the work may be split at other places)
    for bad in ([0, n, n - 1, 3 * n], [0, n, 5 * n, 3 * n], [1, n, 2 * n, 3 * n], [0, n, 2 * n, 3 * n + 2], [-9, n, 2 * n, 3 * n]):
        word, got = flagged(starts=np.array(bad, np.int32))
        assert word & L.LORA_DEV_BAD_SEGMENTS


def test_attention_on_another_stream_and_under_capture():
    c = C.Attention(13, I.BF16, [(1, 500), (1, 3000)], 8, 2, 128, 16)
    ref = run_attention(c)
    kd, vd, q = C.device(c.k, c.dtype), C.device(c.v, c.dtype), C.device(c.q, c.dtype)
    kv = L.KvPages(L.LORA_BF16, kd, vd, c.n_pages, c.page, c.n_kv, c.d)
    out = torch.zeros_like(q)
    ws = torch.empty(max(16, L.lora_tree_attention_workspace_size(kv, c.n_q, c.S, c.T)), dtype=torch.uint8, device="cuda")
    starts, lens, table = cuda(c.starts), cuda(c.lens), cuda(c.table)

    def call():
        L.lora_tree_attention(kv, q, c.n_q, starts, c.S, c.T, lens, table, c.max_pages, None, 0, c.scale, out, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    assert np.array_equal(host(out), ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(host(out), ref)


def test_attention_refusals():
    kd = torch.zeros((4, 2, 8, 16), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((3, 4 * 16), dtype=torch.bfloat16, device="cuda")
    i32 = torch.zeros(8, dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    mask = torch.zeros((3, 1), dtype=torch.int64, device="cuda")

    def status(dtype=L.LORA_BF16, page=8, d=16, q=q, n_q=4, starts=i32, S=2, T=3, lens=i32, table=i32, max_pages=4, mask=mask, words=1,
               out=q, ws=ws, ws_bytes=None, scale=1.0):
        kv = L.KvPages(dtype, kd, kd, 4, 8, 2, 16)
        kv.page_size, kv.head_dim = page, d
        n = L.lora_launch_count()
        try:
            L.lora_tree_attention(kv, q, n_q, starts, S, T, lens, table, max_pages, mask, words, scale, out, ws, ws_bytes=ws_bytes or ws.numel())
        except L.LoraError as e:
            assert L.lora_launch_count() == n
            return e.status
        return 0

    assert status(S=0, T=0) == 0 and status(T=0) == 0
    assert status(dtype=2) == L.LORA_ERR_ARG
    assert status(page=3) == L.LORA_ERR_SHAPE
    assert status(d=20) == L.LORA_ERR_SHAPE
    assert status(n_q=3) == L.LORA_ERR_SHAPE
    assert status(n_q=0) == L.LORA_ERR_SHAPE
    assert status(S=0) == L.LORA_ERR_ARG
    assert status(T=-1) == L.LORA_ERR_ARG
    assert status(q=None) == L.LORA_ERR_ARG
    assert status(starts=None) == L.LORA_ERR_ARG
    assert status(lens=None) == L.LORA_ERR_ARG
    assert status(table=None) == L.LORA_ERR_ARG
    assert status(max_pages=0) == L.LORA_ERR_ARG
    assert status(words=0) == L.LORA_ERR_ARG
    assert status(scale=0.0) == L.LORA_ERR_ARG
    assert status(scale=float("nan")) == L.LORA_ERR_ARG
    assert status(out=None) == L.LORA_ERR_ARG
    assert status(ws_bytes=16) == L.LORA_ERR_ARG
    assert status(max_pages=1 << 30) == L.LORA_ERR_SHAPE


# ----------------------------------------------------------------------------
# fp32 attention of few rows a request on average (requests, n_q, n_kv, d, page, mask)
# ----------------------------------------------------------------------------
FEW_CASES = [
    ([(1, 1)] * 3 + [(1, 64), (1, 65), (1, 4), (1, 3)], 3, 3, 8, 1, None),
    ([(1, n) for n in (1, 31, 32, 33, 63, 64, 65, 127, 500)], 8, 1, 40, 8, None),
    ([(40, 300)] + [(1, 20 + i) for i in range(30)], 2, 1, 72, 16, "tree"),       # one request of many row tiles
    ([(17, 17), (0, 90)] + [(1, 1000 + i) for i in range(12)], 4, 4, 128, 1024, "random"),
    ([(2, 700), (3, 64), (1, 1)], 6, 2, 136, 32, "tree"),
    ([(5, 9), (1, 260), (1, 12)], 4, 2, 200, 4, "tree"),
    ([(2, 3000)], 4, 1, 256, 64, "random"),
    ([(1, 9000 - 37 * i) for i in range(40)], 2, 2, 64, 128, None)]


@pytest.mark.parametrize("case", range(len(FEW_CASES)))
def test_attention_few_rows(case):
    requests, n_q, n_kv, d, page, mask = FEW_CASES[case]
    check_attention(C.Attention(300 + case, I.F32, requests, n_q, n_kv, d, page, mask=mask))


@pytest.mark.parametrize("d", [64, 80, 128, 256])
def test_attention_few_rows_infinite_keys(d):
    """Keys of the prefix that score -infinity drop out; of +infinity or NaN make their rows NaN."""
    c = C.Attention(320, I.F32, [(1, 50), (1, 200), (1, 90)], 2, 2, d, 16)
    c.q[...] = np.abs(c.q) + np.float32(0.5)
    k = c.k.copy()
    k[c.table[1, 0], :, 3, d - 1] = -np.inf             # request 1, token 3
    got = run_attention(c, k=k)
    without = c.k.copy()
    without[c.table[1, 0], :, 3] = -1e30
    assert np.array_equal(got, run_attention(c, k=without)) and np.isfinite(got).all()
    k[c.table[1, 0], :, 3, d - 1] = np.inf
    k[c.table[2, 0], :, 5, 0] = np.nan
    got, clean = run_attention(c, k=k), run_attention(c)
    assert np.array_equal(got[0], clean[0]) and np.isnan(got[1:]).all()
