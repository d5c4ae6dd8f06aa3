"""Variants of the decode-step kernels that a rule on sizes picks and that no other test reaches, against the float64
definitions (bounds: tests/decode_cases.py)."""
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
from tests.test_decode_gpu import (CODE, TORCH, append_bound, append_case, assert_within, check_attention, cuda, host,  # noqa: E402
                                   run_append, run_attention)

# ----------------------------------------------------------------------------
# bf16 attention over pages of 1, 2 and 4 tokens (no tensor copies)
# ----------------------------------------------------------------------------
SMALL_PAGES = [   # requests, n_q, n_kv, d, page, mask
    # tcgen05, units of up to 128 rows
    ([(16, 300), (9, 9), (20, 777), (0, 40), (16, 131)], 8, 2, 64, 1, "tree"),
    ([(16, 300), (9, 9), (20, 777), (16, 128)], 8, 2, 128, 2, "tree"),
    ([(25, 1500) if i % 4 == 0 else (9, 9 + i % 90) for i in range(60)], 8, 2, 64, 4, "random"),
    ([(25, 1500) if i % 4 == 0 else (9, 9 + i % 90) for i in range(60)], 8, 2, 128, 1, "tree"),
    # of up to 256 rows
    ([(64, 700), (33, 1500), (50, 50)], 16, 2, 64, 2, "tree"),
    ([(64, 700), (33, 1500), (50, 50)], 16, 2, 128, 4, "random"),
    ([(70, 300 + i) if i % 2 else (6, 90 + i) for i in range(40)], 16, 4, 128, 1, None),
    # warp MMAs
    ([(1, 300), (1, 17), (1, 1), (1, 2000)], 8, 8, 128, 4, None),
    ([(3, 300), (1, 64), (2, 1000)], 8, 2, 80, 2, "tree"),
    ([(3, 300), (1, 65), (2, 1000)], 4, 2, 72, 1, "tree"),
    ([(2, 333), (6, 500)], 8, 1, 256, 1, "tree"),
    ([(40, 300), (20, 90)], 8, 2, 192, 4, "random")]


@pytest.mark.parametrize("case", range(len(SMALL_PAGES)))
def test_attention_small_pages(case):
    requests, n_q, n_kv, d, page, mask = SMALL_PAGES[case]
    check_attention(C.Attention(500 + case, I.BF16, requests, n_q, n_kv, d, page, mask=mask))


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("heads, d, page", [((4, 4), 64, 1), ((4, 4), 128, 2), ((8, 2), 128, 4), ((8, 2), 64, 2), ((32, 2), 64, 4),
                                            ((32, 2), 128, 1), ((8, 4), 80, 2), ((8, 4), 256, 4)])
def test_attention_small_pages_non_finite_drafts(bad, heads, d, page):
    c = C.Attention(8, I.BF16, [(20, 83), (9, 9), (8, 40)], *heads, d, page, mask="tree")
    clean = run_attention(c)
    k, v = c.k.copy(), c.v.copy()
    j = 3
    for s in range(3):                                   # drafted token 3 of every request holds bad values
        at = int(c.lens[s]) - (int(c.starts[s + 1]) - int(c.starts[s])) + j
        v[c.table[s, at // page], :, at % page] = bad
        if s:
            k[c.table[s, at // page], :, at % page] = bad
    got = run_attention(c, k=k, v=v)
    see = np.concatenate([m[:, j] for m in c.masks])
    assert np.array_equal(got[~see], clean[~see])
    assert see.any() and not np.isfinite(got[:20][see[:20]]).any()


@pytest.mark.parametrize("n_q", [8, 32])
@pytest.mark.parametrize("page", [1, 4])
def test_attention_small_pages_in_place_and_bad_pages(n_q, page):
    c = C.Attention(12, I.BF16, [(16, 90), (16, 70), (16, 200)], n_q, 2, 64, page, mask="tree", garbage=0.0)
    good = run_attention(c)
    assert np.array_equal(run_attention(c, out="q"), good)
    table = c.table.copy()
    table[1, 2], table[1, 3] = c.n_pages, -3
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_attention(c, status, table=table)
    assert int(status) == L.LORA_DEV_BAD_PAGE
    keep = np.r_[0:16, 32:48]
    assert np.array_equal(got[keep], good[keep])


# ----------------------------------------------------------------------------
# Append, neighbouring pairs: three heads a thread (more than 1000 blocks of one in bf16, 16000 in fp32, and more than one
# block a token), and the sizes beside that
# ----------------------------------------------------------------------------
MANY_HEADS = [   # T, n_q, n_kv, d, rot, page, interleaved, norm, fused
    (800, 28, 4, 128, 128, 16, True, True, True), (1600, 5, 1, 64, 32, 64, True, False, False), (400, 33, 11, 256, 128, 8, True, True, False),
    (1001, 16, 8, 80, 80, 1, True, True, True), (1501, 0, 3, 128, 8, 32, True, True, False),
    (1000, 28, 4, 64, 64, 16, True, True, False), (801, 0, 9, 128, 8, 4, True, True, False), (8201, 14, 2, 128, 8, 16, True, True, False)]


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("case", MANY_HEADS, ids=lambda c: "-".join(map(str, c)))
def test_kv_append_many_heads(case, dtype):
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
    if not fused and n_q:
        again = run_append(case, dtype, arrays, in_place=True)
        assert np.array_equal(again[0], got[0]) and np.array_equal(again[1], got[1])


# ----------------------------------------------------------------------------
# 4-bit products: more rows than one turn of the blocks, wide projections without a cluster, non-finite activations
# ----------------------------------------------------------------------------
W4_TALL = [   # T, h_in, h_out, group
    (12, 2080, 1900, 32), (12, 2048, 2048, 128), (64, 2112, 2400, 64), (33, 2048, 4600, 128), (16, 2048, 4800, 64),   # clusters of 8, 4, 2
    (1, 512, 20001, 64), (8, 256, 39000, 128), (3, 288, 19600, 32), (5, 4224, 19500, 128),            # warp MMAs, more than one turn
    (9, 1024, 9800, 128), (24, 1056, 9999, 32), (64, 1088, 9801, 64), (40, 640, 20000, 128),          # tcgen05, no cluster
    (1, 14336, 300, 64), (3, 14336, 300, 64), (6, 13312, 2500, 128), (7, 13312, 2500, 32)]            # x in parts; both kernels


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("case", W4_TALL, ids=lambda c: "-".join(map(str, c)))
def test_w4_tall(case, dtype):
    T, h_in, h_out, group = case
    x, codes, scales, z = C.w4_case(sum(case), dtype, T, h_in, h_out, group, True)
    ref, mag = D.w4_matvec(x, codes, scales, z, group)
    args = (CODE[dtype], C.device(x, dtype), T, h_in, cuda(codes), cuda(scales).to(torch.bfloat16), cuda(z), group, h_out)
    y = torch.full((T, h_out), float("nan"), dtype=TORCH[dtype], device="cuda")
    L.lora_w4_matvec(*args, y)
    assert_within(host(y), ref, C.w4_bound(ref, mag, h_in, group, dtype))
    for _ in range(3):
        again = torch.full_like(y, float("nan"))
        L.lora_w4_matvec(*args, again)
        assert torch.equal(again, y)


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("T", [12, 20, 40, 66])
def test_w4_non_finite_activations_of_many_tokens(T, dtype):
    x, codes, scales, z = C.w4_case(6, dtype, T, 1088, 200, 64, False)
    codes[:] = 0x99                                      # codes less zeros are 1: infinities keep their sign
    x[1, 5], x[2, 1087], x[T - 1, 640], x[T - 2, 700] = np.nan, np.inf, -np.inf, np.nan
    y = torch.empty((T, 200), dtype=TORCH[dtype], device="cuda")
    L.lora_w4_matvec(CODE[dtype], C.device(x, dtype), T, 1088, cuda(codes), cuda(scales).to(torch.bfloat16), None, 64, 200, y)
    y = host(y)
    others = np.setdiff1d(np.arange(T), [1, 2, T - 1, T - 2])
    assert np.isfinite(y[others]).all() and np.isnan(y[[1, T - 2]]).all() and np.isposinf(y[2]).all() and np.isneginf(y[T - 1]).all()


# ----------------------------------------------------------------------------
# Infinite values that every row sees come out infinite, and stay in their column
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("requests, n_q, n_kv, d, page", [
    ([(1, 300), (1, 70)], 4, 2, 128, 16), ([(2, 300), (3, 70)], 8, 2, 80, 4), ([(20, 500), (16, 90)], 8, 2, 64, 16),
    ([(20, 500), (16, 90)], 8, 2, 128, 2), ([(60, 700), (40, 90)], 16, 2, 128, 64)])
def test_attention_infinite_values_of_the_prefix(requests, n_q, n_kv, d, page, dtype):
    c = C.Attention(600, dtype, requests, n_q, n_kv, d, page, mask="tree", scale=0.02)      # no probability underflows
    clean = run_attention(c)
    v = c.v.copy()
    for s, (at, col, value) in enumerate(((37, 5, np.inf), (3, d - 1, -np.inf))):
        v[c.table[s, at // page], :, at % page, col] = value
    got = run_attention(c, v=v)
    first = requests[0][0]
    expected = clean.reshape(-1, n_q, d).copy()
    expected[:first, :, 5], expected[first:, :, d - 1] = np.inf, -np.inf
    assert np.array_equal(got.reshape(-1, n_q, d), expected)
