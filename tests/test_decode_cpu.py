"""Host-side checks of the decode-step calls: arguments are refused before any
launch, sizes are computed, and empty calls succeed, all without a GPU (the
pointers are host memory that nothing reads)."""
import ctypes

import pytest

from segmented_gathered_rank_gb300 import lora as L

BF16, F32 = L.LORA_BF16, L.LORA_F32
BUF = ctypes.create_string_buffer(1 << 16)
P = (ctypes.addressof(BUF) + 255) & ~255


def pages(**change):
    kv = L.KvPages.__new__(L.KvPages)          # the struct without tensors
    for name, value in dict(dict(dtype=BF16, k=P, v=P, n_pages=64, page_size=16, n_kv_heads=2, head_dim=128,
                                 status=None), **change).items():
        setattr(kv, name, value)
    return kv


def w4(dtype=BF16, x=P, T=4, h_in=256, codes=P, scales=P, zeros=None, group=64, h_out=32, y=P):
    return L._lib.lora_w4_matvec(dtype, x, T, h_in, codes, scales, zeros, group, h_out, y, None)


@pytest.mark.parametrize("change, code", [
    (dict(dtype=7), L.LORA_ERR_ARG), (dict(T=-1), L.LORA_ERR_ARG), (dict(h_in=0), L.LORA_ERR_ARG),
    (dict(h_out=-5), L.LORA_ERR_ARG), (dict(group=48), L.LORA_ERR_SHAPE), (dict(h_in=200), L.LORA_ERR_SHAPE),
    (dict(x=P + 2), L.LORA_ERR_ARG), (dict(codes=P + 8), L.LORA_ERR_ARG), (dict(y=P + 4), L.LORA_ERR_ARG),
    (dict(scales=P + 1), L.LORA_ERR_ARG), (dict(x=None), L.LORA_ERR_ARG), (dict(scales=None), L.LORA_ERR_ARG)])
def test_w4_matvec_refuses(change, code):
    assert w4(**change) == code


def test_w4_matvec_without_tokens():
    before = L.lora_launch_count()
    assert w4(T=0, x=None, y=None) == L.LORA_OK
    assert L.lora_launch_count() == before


BAD_PAGES = [
    (dict(dtype=3), L.LORA_ERR_ARG), (dict(k=None), L.LORA_ERR_ARG), (dict(v=P + 8), L.LORA_ERR_ARG),
    (dict(status=P + 2), L.LORA_ERR_ARG), (dict(n_pages=0), L.LORA_ERR_ARG), (dict(n_kv_heads=0), L.LORA_ERR_ARG),
    (dict(page_size=24), L.LORA_ERR_SHAPE), (dict(page_size=2048), L.LORA_ERR_SHAPE),
    (dict(head_dim=12), L.LORA_ERR_SHAPE), (dict(head_dim=264), L.LORA_ERR_SHAPE),
    (dict(n_pages=1 << 26, page_size=16), L.LORA_ERR_SHAPE)]      # 2^26 * 16 * 2 rows


def append(kv, q=P, ld_q=512, k=P, ld_k=256, v=P, ld_v=256, T=3, n_q=4, positions=P, slots=P, cos_sin=P, n_pos=16,
           rot=128, interleaved=False, q_norm=None, k_norm=None, eps=1e-6, q_out=P):
    return L._lib.lora_kv_append(ctypes.byref(kv), q, ld_q, k, ld_k, v, ld_v, T, n_q, positions, slots, cos_sin, n_pos,
                                 rot, int(interleaved), q_norm, k_norm, eps, q_out, None)


@pytest.mark.parametrize("change, code", BAD_PAGES)
def test_append_refuses_pages(change, code):
    assert append(pages(**change)) == code


@pytest.mark.parametrize("change, code", [
    (dict(T=-1), L.LORA_ERR_ARG), (dict(rot=-2), L.LORA_ERR_ARG), (dict(eps=-1.0), L.LORA_ERR_ARG),
    (dict(eps=float("nan")), L.LORA_ERR_ARG), (dict(rot=130), L.LORA_ERR_SHAPE), (dict(rot=7), L.LORA_ERR_SHAPE),
    (dict(n_q=3), L.LORA_ERR_SHAPE), (dict(ld_k=255), L.LORA_ERR_SHAPE), (dict(ld_v=260), L.LORA_ERR_SHAPE),
    (dict(ld_q=504), L.LORA_ERR_SHAPE), (dict(slots=P + 4), L.LORA_ERR_ARG), (dict(slots=None), L.LORA_ERR_ARG),
    (dict(q_out=None), L.LORA_ERR_ARG), (dict(positions=None), L.LORA_ERR_ARG), (dict(n_pos=0), L.LORA_ERR_ARG),
    (dict(cos_sin=None), L.LORA_ERR_ARG), (dict(q_norm=P + 4), L.LORA_ERR_ARG),
    (dict(ld_q=1024), L.LORA_ERR_ARG)])       # in place, rows apart
def test_append_refuses(change, code):
    assert append(pages(), **change) == code


def attend(kv, q=P, n_q=4, starts=P, S=2, T=2, lens=P, table=P, max_pages=4, mask=None, words=0, scale=0.1, out=P,
           workspace=P, ws_bytes=1 << 30):
    return L._lib.lora_tree_attention(ctypes.byref(kv), q, n_q, starts, S, T, lens, table, max_pages, mask, words, scale,
                                      out, workspace, ws_bytes, None)


@pytest.mark.parametrize("change, code", BAD_PAGES)
def test_attention_refuses_pages(change, code):
    kv = pages(**change)
    assert attend(kv) == code
    assert L._lib.lora_tree_attention_workspace_size(ctypes.byref(kv), 4, 2, 2) == 0


@pytest.mark.parametrize("change, code", [
    (dict(n_q=0), L.LORA_ERR_SHAPE), (dict(n_q=5), L.LORA_ERR_SHAPE), (dict(scale=0.0), L.LORA_ERR_ARG),
    (dict(scale=-1.0), L.LORA_ERR_ARG), (dict(scale=float("inf")), L.LORA_ERR_ARG), (dict(S=-1), L.LORA_ERR_ARG),
    (dict(S=0), L.LORA_ERR_ARG), (dict(T=-1), L.LORA_ERR_ARG), (dict(max_pages=-1), L.LORA_ERR_ARG),
    (dict(max_pages=0), L.LORA_ERR_ARG), (dict(mask=P), L.LORA_ERR_ARG), (dict(mask=P + 4, words=1), L.LORA_ERR_ARG),
    (dict(max_pages=1 << 28), L.LORA_ERR_SHAPE), (dict(T=1 << 30), L.LORA_ERR_SHAPE), (dict(q=None), L.LORA_ERR_ARG),
    (dict(out=P + 8), L.LORA_ERR_ARG), (dict(workspace=P + 4), L.LORA_ERR_ARG), (dict(lens=P + 2), L.LORA_ERR_ARG)])
def test_attention_refuses(change, code):
    assert attend(pages(), **change) == code


def test_attention_without_tokens():
    before = L.lora_launch_count()
    assert attend(pages(), T=0, S=0, q=None, out=None, workspace=None) == L.LORA_OK
    assert L.lora_launch_count() == before


def test_device_status_bits_are_distinct():
    bits = [v for n, v in vars(L).items() if n.startswith("LORA_DEV_") and isinstance(v, int) and v]
    assert len(bits) == len(set(bits)) and all(b & (b - 1) == 0 for b in bits)


def test_append_without_tokens():
    before = L.lora_launch_count()
    assert append(pages(), T=0, q=None, k=None, v=None, slots=None, q_out=None) == L.LORA_OK
    assert L.lora_launch_count() == before


def test_pages_want_their_size():
    class Tensor:
        def numel(self):
            return 100

    with pytest.raises(ValueError):
        L.KvPages(BF16, Tensor(), Tensor(), 64, 16, 2, 128)
