"""Decode-step operators on the GPU where units, tables and sizes meet (definitions: oracle/decode.py; bounds:
tests/decode_cases.py)."""
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
from tests.test_decode_gpu import CODE, TORCH, assert_within, check_attention, cuda, host, run_attention  # noqa: E402


# ----------------------------------------------------------------------------
# tcgen05 attention: units in which only one softmax stream has a part, in turn with units in which both have
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("requests", [
    [(16, 30 + i) if i % 2 else (16, 700 + 40 * (i % 7)) for i in range(100)],     # one key tile, then several: 64 rows a unit
    [(9, 9 + i % 90) if i % 4 else (25, 1500) for i in range(140)],                # three units of one tile in a row
    [(6, 90 + i) if i % 2 else (70, 300 + i) for i in range(100)],                 # 24 rows a unit, then 256 and 24
], ids=["one_tile", "one_tile_runs", "few_rows"])
def test_attention_streams_take_turns(requests, d):
    c = C.Attention(400 + d, I.BF16, requests, 16, 4, d, 16, mask="tree")
    got = check_attention(c)
    for _ in range(10):
        assert np.array_equal(run_attention(c), got)


# ----------------------------------------------------------------------------
# Segments that overlap: T tokens counted again and again
# ----------------------------------------------------------------------------
def overlapping(dtype, T, S, n_q, n_kv, d, page, max_pages, guard=4096):
    """seg_starts 0, T, 0, T, ..: (status word, whether out was written, whether the bytes after the workspace were)."""
    dt = torch.bfloat16 if dtype == I.BF16 else torch.float32
    k, v = (torch.randn(4, n_kv, page, d, device="cuda").to(dt) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = L.KvPages(L.LORA_BF16 if dtype == I.BF16 else L.LORA_F32, k, v, 4, page, n_kv, d, status=status)
    q = torch.randn(T, n_q * d, device="cuda").to(dt)
    out = torch.full_like(q, float("nan"))
    starts = torch.tensor([0, T] * (S // 2) + [0], dtype=torch.int32, device="cuda")
    lens = torch.full((S,), max_pages * page, dtype=torch.int32, device="cuda")
    table = torch.zeros((S, max_pages), dtype=torch.int32, device="cuda")
    size = L.lora_tree_attention_workspace_size(kv, n_q, S, T)
    ws = torch.full((size + guard,), 0xAB, dtype=torch.uint8, device="cuda")
    L.lora_tree_attention(kv, q, n_q, starts, S, T, lens, table, max_pages, None, 0, 0.1, out, ws, ws_bytes=size)
    torch.cuda.synchronize()
    return int(status), not bool(torch.isnan(out).all()), not bool((ws[size:] == 0xAB).all())


@pytest.mark.parametrize("dtype, T, S, d", [(I.BF16, 32, 64, 64), (I.BF16, 128, 16, 128), (I.BF16, 512, 16, 64), (I.F32, 32, 64, 128),
                                            (I.F32, 512, 16, 64)])
def test_attention_overlapping_segments_compute_nothing(dtype, T, S, d):
    assert overlapping(dtype, T, S, 8, 1, d, 64, 8) == (L.LORA_DEV_BAD_SEGMENTS, False, False)


@pytest.mark.parametrize("T, S", [(2048, 2048), (8192, 2048)])
def test_attention_overlapping_segments_beyond_32_bits_of_places(T, S):
    """The places that these tables name pass 2^32."""
    assert overlapping(I.BF16, T, S, 32, 8, 64, 1024, 128) == (L.LORA_DEV_BAD_SEGMENTS, False, False)


# ----------------------------------------------------------------------------
# 4-bit products on tcgen05: many tiles of weights through the stages of tensor memory
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("T, h_in, h_out, group", [(40, 8192, 1300, 128), (12, 16384, 300, 64), (24, 12320, 640, 32)])
def test_w4_stages_of_long_rows(T, h_in, h_out, group, dtype):
    x, codes, scales, z = C.w4_case(T + h_in, dtype, T, h_in, h_out, group, True)
    ref, mag = D.w4_matvec(x, codes, scales, z, group)
    args = (CODE[dtype], C.device(x, dtype), T, h_in, cuda(codes), cuda(scales).to(torch.bfloat16), cuda(z), group, h_out)
    y = torch.full((T, h_out), float("nan"), dtype=TORCH[dtype], device="cuda")
    L.lora_w4_matvec(*args, y)
    assert_within(host(y), ref, C.w4_bound(ref, mag, h_in, group, dtype))
    for _ in range(20):
        again = torch.full_like(y, float("nan"))
        L.lora_w4_matvec(*args, again)
        assert torch.equal(again, y)


# ----------------------------------------------------------------------------
# A workspace made once for the largest batch
# ----------------------------------------------------------------------------
def pages_of(dtype, n_kv, d, page=16, n_pages=40):
    k, v = (torch.randn(n_pages, n_kv, page, d, device="cuda").to(TORCH[dtype]) for _ in range(2))
    return L.KvPages(CODE[dtype], k, v, n_pages, page, n_kv, d)


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("d", [64, 80, 128, 256])
def test_workspace_of_the_largest_batch_serves_every_smaller_one(dtype, d):
    for group in (1, 4, 16):
        kv = pages_of(dtype, 2, d)
        most = L.lora_tree_attention_workspace_size(kv, 2 * group, 128, 128)
        ws = torch.empty(most, dtype=torch.uint8, device="cuda")
        for T in (1, 2, 7, 16, 33, 64, 127, 128):
            for S in {1, 2, (T + 15) // 16, (T + 1) // 2, T} - {t for t in (1, 2) if t > T}:
                assert L.lora_tree_attention_workspace_size(kv, 2 * group, S, T) <= most
                starts = torch.linspace(0, T, S + 1, device="cuda").round().int()
                lens = (starts[1:] - starts[:-1] + 3).int()
                table = torch.arange(9, device="cuda", dtype=torch.int32).repeat(S, 1)
                q = torch.randn(T, 2 * group * d, device="cuda").to(TORCH[dtype])
                out, own = torch.zeros_like(q), torch.zeros_like(q)
                size = L.lora_tree_attention_workspace_size(kv, 2 * group, S, T)
                for o, w in ((out, ws), (own, torch.empty(size, dtype=torch.uint8, device="cuda"))):
                    L.lora_tree_attention(kv, q, 2 * group, starts, S, T, lens, table, 9, None, 0, 0.1, o, w)
                assert torch.equal(out, own) and bool(torch.isfinite(out.float()).all())
