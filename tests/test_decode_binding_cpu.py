"""The Python side of the decode-step calls without a GPU: what their objects keep alive and what they pass on."""
import ctypes
import gc
import math
import weakref

import pytest

from segmented_gathered_rank_gb300 import lora as L

BUF = ctypes.create_string_buffer(1 << 16)
P = (ctypes.addressof(BUF) + 255) & ~255


class Cuda:
    """Stands in for a CUDA tensor: host memory that nothing reads."""
    is_cuda = True

    def __init__(self, *shape, stride=None):
        self.shape, self._stride = shape, stride or tuple(math.prod(shape[i + 1:]) for i in range(len(shape)))

    def numel(self):
        return math.prod(self.shape)

    def dim(self):
        return len(self.shape)

    def stride(self, i):
        return self._stride[i]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return P


def test_pages_let_their_tensors_go():
    """No cycle: a cache of many GB is free as soon as the last reference to it is."""
    k, v = Cuda(4, 2, 8, 16), Cuda(4, 2, 8, 16)
    kv = L.KvPages(L.LORA_BF16, k, v, 4, 8, 2, 16)
    assert L.lora_tree_attention_workspace_size(kv, 4, 0, 0) == 16       # the struct as the library reads it
    alive = weakref.ref(k), weakref.ref(v)
    del k, v
    assert all(a() is not None for a in alive)
    gc.disable()
    try:
        del kv
        assert all(a() is None for a in alive)
    finally:
        gc.enable()


def append_status(monkeypatch, q, k, v, T, n_q=4, slots=None):
    """What lora_kv_append returns without launching: n_pos 0 is refused last, once the row strides have passed."""
    got = []
    monkeypatch.setattr(L, "_check", lambda rc, where: got.append(rc))
    kv = L.KvPages(L.LORA_BF16, Cuda(4, 2, 8, 16), Cuda(4, 2, 8, 16), 4, 8, 2, 16)
    L.lora_kv_append(kv, q, k, v, T, n_q, Cuda(T), Cuda(T), Cuda(1, 16), 0, 16, False, Cuda(T, n_q * 16), stream=0)
    return got[0]


def test_append_takes_one_row_of_any_stride(monkeypatch):
    """(W @ x.T).T of one token has the shape [1, width] and the strides (1, 1)."""
    one = [Cuda(1, w, stride=(1, 1)) for w in (64, 32, 32)]
    assert append_status(monkeypatch, *one, T=1) == L.LORA_ERR_ARG       # for n_pos, not LORA_ERR_SHAPE for the rows
    two = [Cuda(2, w, stride=(8, 1)) for w in (64, 32, 32)]
    assert append_status(monkeypatch, *two, T=2) == L.LORA_ERR_SHAPE     # rows that overlap


def test_append_refuses_rows_further_apart_than_an_int(monkeypatch):
    k = Cuda(2, 32)
    for far in (1 << 31, (1 << 32) + 64):           # the second would wrap to a valid distance
        with pytest.raises(ValueError, match="an int"):
            append_status(monkeypatch, Cuda(2, 64, stride=(far, 1)), k, k, T=2)


@pytest.mark.parametrize("T", [1, 8, 9, 64])
@pytest.mark.parametrize("h_in, h_out", [(64, (1 << 31) - 1), (64, (1 << 31) - (1 << 16) + 1), ((1 << 31) - 64, 32)])
def test_w4_refuses_sizes_that_indexes_would_pass(T, h_in, h_out):
    before = L.lora_launch_count()
    assert L._lib.lora_w4_matvec(L.LORA_BF16, P, T, h_in, P, P, None, 64, h_out, P, None) == L.LORA_ERR_SHAPE
    assert L.lora_launch_count() == before
