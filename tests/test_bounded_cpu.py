"""Host-side checks of the calls of a bounded cache: refused before any launch, without a GPU (the pointers are host
memory that nothing reads)."""
import ctypes
import re

import numpy as np
import pytest

from segmented_gathered_rank_gb300 import lora as L
from tests.test_decode_binding_cpu import Cuda as Whole
from tests.test_decode_cpu import BAD_PAGES, P, pages

AXES = bytes(i % 3 for i in range(64))


class Cuda(Whole):
    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]


def call(name, kv, layout, *values):
    return getattr(L._lib, name)(ctypes.addressof(kv), layout.pack(*(0 if v is None else v for v in values)), None)


def axes(kv, q=P, ld_q=512, k=P, ld_k=256, v=P, ld_v=256, T=3, n_q=4, positions=P, n_axes=3, pair_axis=AXES, slots=P, cos_sin=P,
         n_pos=16, rot=128, interleaved=False, q_norm=None, k_norm=None, eps=1e-6, q_out=P):
    return call("lora_kv_append_axes", kv, L._AXES, q, k, v, q_out, positions, slots, cos_sin, q_norm, k_norm, ld_q, ld_k, ld_v, T, n_q,
                n_axes, n_pos, rot, int(interleaved), eps, pair_axis)


@pytest.mark.parametrize("change, code", BAD_PAGES)
def test_append_axes_refuses_pages(change, code):
    assert axes(pages(**change)) == code


@pytest.mark.parametrize("change, code", [
    (dict(n_axes=0), L.LORA_ERR_ARG), (dict(n_axes=L.LORA_MAX_AXES + 1), L.LORA_ERR_ARG),
    (dict(n_axes=2), L.LORA_ERR_ARG), (dict(pair_axis=bytes(63) + bytes([3])), L.LORA_ERR_ARG),        # an axis beyond n_axes
    (dict(T=0, n_axes=2), L.LORA_ERR_ARG),
    (dict(T=-1), L.LORA_ERR_ARG), (dict(rot=-2), L.LORA_ERR_ARG), (dict(eps=-1.0), L.LORA_ERR_ARG),
    (dict(eps=float("nan")), L.LORA_ERR_ARG), (dict(rot=130), L.LORA_ERR_SHAPE), (dict(rot=7), L.LORA_ERR_SHAPE),
    (dict(n_q=3), L.LORA_ERR_SHAPE), (dict(ld_k=255), L.LORA_ERR_SHAPE), (dict(ld_v=260), L.LORA_ERR_SHAPE),
    (dict(ld_q=504), L.LORA_ERR_SHAPE), (dict(slots=P + 4), L.LORA_ERR_ARG), (dict(slots=None), L.LORA_ERR_ARG),
    (dict(q_out=None), L.LORA_ERR_ARG), (dict(positions=None), L.LORA_ERR_ARG), (dict(positions=P + 2), L.LORA_ERR_ARG),
    (dict(n_pos=0), L.LORA_ERR_ARG), (dict(cos_sin=None), L.LORA_ERR_ARG), (dict(k_norm=P + 4), L.LORA_ERR_ARG),
    (dict(ld_q=1024), L.LORA_ERR_ARG)])       # in place, rows apart
def test_append_axes_refuses(change, code):
    before = L.lora_launch_count()
    assert axes(pages(), **change) == code
    assert L.lora_launch_count() == before


def test_append_axes_without_tokens():
    before = L.lora_launch_count()
    assert axes(pages(), T=0, q=None, k=None, v=None, q_out=None, positions=None, slots=None) == L.LORA_OK
    assert L.lora_launch_count() == before


def test_no_arguments():
    kv = pages()
    for name in ("lora_kv_append_axes", "lora_tree_attention_weights", "lora_kv_evict"):
        assert getattr(L._lib, name)(ctypes.addressof(kv), None, None) == L.LORA_ERR_ARG


def test_packed_structs_are_the_header_s(tmp_path):
    """Field by field, as the compiler lays them out."""
    import os
    import shutil
    import subprocess
    if not shutil.which("gcc"):
        pytest.skip("no C compiler")
    layouts = {"lora_append_axes": (L._AXES, "q k v q_out positions slots cos_sin q_norm k_norm ld_q ld_k ld_v T n_q_heads n_axes n_pos rot_dim "
                                             "interleaved eps pair_axis"),
               "lora_attention_weights": (L._WEIGHTS, "weights q seg_starts kv_lens page_table tree_mask out workspace ws_bytes n_q_heads S T "
                                                      "max_pages mask_words scale decay"),
               "lora_eviction": (L._EVICTION, "scores weights kv_lens page_table keep kept new_lens S max_pages first recent ld_kept")}
    lines = [f'printf("{name} %zu", sizeof({name}));' + "".join(f'printf(" %zu", offsetof({name}, {f}));' for f in fields.split()) + 'puts("");'
             for name, (_, fields) in layouts.items()]
    source = tmp_path / "offsets.c"
    source.write_text('#include <stdio.h>\n#include "lora.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0;\n}\n")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-I", include, "-o", str(tmp_path / "offsets"), str(source)], check=True)
    got = {line.split()[0]: [int(x) for x in line.split()[1:]]
           for line in subprocess.run([str(tmp_path / "offsets")], capture_output=True, text=True, check=True).stdout.splitlines()}
    sizes = {"P": 8, "N": 8, "i": 4, "f": 4}
    for name, (layout, fields) in layouts.items():
        at, offsets = 0, []
        for count, kind in re.findall(r"(\d*)([PNifsx])", layout.format.lstrip("@")):
            if kind in "sx":
                offsets += [at] if kind == "s" else []
                at += int(count)
                continue
            for _ in range(int(count or 1)):
                at = -(-at // sizes[kind]) * sizes[kind]
                offsets.append(at)
                at += sizes[kind]
        assert got[name] == [layout.size, *offsets] and len(offsets) == len(fields.split())


def test_pair_axis_from_python(monkeypatch):
    """Whole numbers of any type; what is too short or not a byte is refused."""
    got = []
    monkeypatch.setattr(L, "_check", lambda rc, where: got.append(rc))
    kv = L.KvPages(L.LORA_BF16, Cuda(4, 2, 8, 16), Cuda(4, 2, 8, 16), 4, 8, 2, 16)

    def call(pair_axis, n_axes=3, n_pos=0):
        got.clear()
        L.lora_kv_append_axes(kv, Cuda(3, 64), Cuda(3, 32), Cuda(3, 32), 3, 4, Cuda(3, n_axes), n_axes, pair_axis, Cuda(3), Cuda(1, 16), n_pos,
                              16, False, Cuda(3, 64), stream=0)
        return got[0] if got else 0

    # n_pos 0 is refused after pair_axis has passed; with n_axes 2 the axis 2 is refused before
    for a in (bytes([0, 1, 2, 0, 1, 2, 0, 1]), [0, 1, 2, 0, 1, 2, 0, 1], np.array([0, 1, 2, 0, 1, 2, 0, 1])):
        assert call(a) == L.LORA_ERR_ARG and call(a, n_axes=2) == L.LORA_ERR_ARG
    with pytest.raises(ValueError):
        call([0, 1, 2])
    with pytest.raises(ValueError):
        call([0, 1, 2, 0, 1, 2, 0, 256])


def evict(kv, scores=P, weights=P, S=2, lens=P + (1 << 14) + 64, table=P + (1 << 14), max_pages=4, keep=P + (1 << 14) + 128,
          first=1, recent=2, kept=P + (1 << 14) + 512, ld=8, new_lens=P + (1 << 14) + 256):
    return call("lora_kv_evict", kv, L._EVICTION, scores, weights, lens, table, keep, kept, new_lens, S, max_pages, first, recent, ld)


@pytest.mark.parametrize("change, code", BAD_PAGES)
def test_evict_refuses_pages(change, code):
    assert evict(pages(**change)) == code


@pytest.mark.parametrize("change, code", [
    (dict(S=-1), L.LORA_ERR_ARG), (dict(max_pages=-1), L.LORA_ERR_ARG), (dict(max_pages=0), L.LORA_ERR_ARG), (dict(first=-1), L.LORA_ERR_ARG),
    (dict(recent=-1), L.LORA_ERR_ARG), (dict(ld=-1), L.LORA_ERR_ARG), (dict(scores=None), L.LORA_ERR_ARG), (dict(lens=None), L.LORA_ERR_ARG),
    (dict(table=None), L.LORA_ERR_ARG), (dict(keep=None), L.LORA_ERR_ARG), (dict(kept=None), L.LORA_ERR_ARG), (dict(new_lens=None), L.LORA_ERR_ARG),
    (dict(scores=P + 2), L.LORA_ERR_ARG), (dict(weights=P + 1), L.LORA_ERR_ARG), (dict(kept=P + 3), L.LORA_ERR_ARG),
    (dict(weights=P + 4), L.LORA_ERR_ARG), (dict(scores=P + 64 * 16 * 2 * 4 - 4), L.LORA_ERR_ARG),       # half over each other
    (dict(new_lens=P + (1 << 14) + 64), L.LORA_ERR_ARG), (dict(new_lens=P + (1 << 14) + 132), L.LORA_ERR_ARG),
    (dict(new_lens=P + (1 << 14) + 124), L.LORA_ERR_ARG), (dict(new_lens=P + (1 << 14) + 28), L.LORA_ERR_ARG),
    (dict(kept=P + (1 << 14)), L.LORA_ERR_ARG), (dict(kept=P + (1 << 14) + 132), L.LORA_ERR_ARG), (dict(kept=P + 64), L.LORA_ERR_ARG),
    (dict(kept=P + (1 << 14) + 260), L.LORA_ERR_ARG),
    (dict(max_pages=1 << 27), L.LORA_ERR_SHAPE), (dict(S=1 << 28), L.LORA_ERR_SHAPE)])
def test_evict_refuses(change, code):
    before = L.lora_launch_count()
    assert evict(pages(), **change) == code
    assert L.lora_launch_count() == before


def test_evict_without_requests():
    before = L.lora_launch_count()
    assert evict(pages(), S=0, scores=None, lens=None, table=None, keep=None, kept=None, new_lens=None) == L.LORA_OK
    assert L.lora_launch_count() == before


def test_planes_that_are_too_small_are_refused_in_python():
    kv = L.KvPages(L.LORA_BF16, Cuda(4, 2, 8, 16), Cuda(4, 2, 8, 16), 4, 8, 2, 16)
    args = (2, Cuda(2), Cuda(2, 4), 4, Cuda(2), 0, 0, Cuda(2, 2, 8), 8, Cuda(2))
    with pytest.raises(ValueError):
        L.lora_kv_evict(kv, Cuda(4, 2, 7), None, *args, stream=0)
    with pytest.raises(ValueError):
        L.lora_kv_evict(kv, Cuda(4, 2, 8), Cuda(63), *args, stream=0)
    with pytest.raises(ValueError):
        L.lora_kv_evict(kv, Cuda(4, 2, 8), None, *args[:7], Cuda(2, 2, 7), 8, Cuda(2), stream=0)


def weigh(kv, weights=P, decay=1.0, q=P, n_q=4, starts=P, S=2, T=2, lens=P, table=P, max_pages=4, mask=None, words=0, scale=0.1, out=P,
          workspace=P, ws_bytes=1 << 30):
    out = P + (1 << 13) if out == P else out
    return call("lora_tree_attention_weights", kv, L._WEIGHTS, weights, q, starts, lens, table, mask, out, workspace, ws_bytes, n_q, S, T,
                max_pages, words, scale, decay)


@pytest.mark.parametrize("change, code", BAD_PAGES)
def test_attention_weights_refuses_pages(change, code):
    kv = pages(**change)
    assert weigh(kv) == code
    assert L._lib.lora_tree_attention_weights_workspace_size(ctypes.byref(kv), 4, 2, 2, 4) == 0


@pytest.mark.parametrize("change, code", [
    (dict(weights=None), L.LORA_ERR_ARG), (dict(weights=P + 4), L.LORA_ERR_ARG), (dict(decay=-0.1), L.LORA_ERR_ARG),
    (dict(decay=1.5), L.LORA_ERR_ARG), (dict(decay=float("nan")), L.LORA_ERR_ARG),
    (dict(n_q=0), L.LORA_ERR_SHAPE), (dict(n_q=5), L.LORA_ERR_SHAPE), (dict(scale=0.0), L.LORA_ERR_ARG),
    (dict(scale=float("inf")), L.LORA_ERR_ARG), (dict(S=-1), L.LORA_ERR_ARG), (dict(S=0), L.LORA_ERR_ARG), (dict(T=-1), L.LORA_ERR_ARG),
    (dict(max_pages=-1), L.LORA_ERR_ARG), (dict(max_pages=0), L.LORA_ERR_ARG), (dict(mask=P), L.LORA_ERR_ARG),
    (dict(mask=P + 4, words=1), L.LORA_ERR_ARG), (dict(q=P + 8), L.LORA_ERR_ARG), (dict(out=None), L.LORA_ERR_ARG),
    (dict(starts=P + 2), L.LORA_ERR_ARG), (dict(lens=None), L.LORA_ERR_ARG), (dict(table=None), L.LORA_ERR_ARG),
    (dict(out=P + 16), L.LORA_ERR_ARG), (dict(out=P + 2 * 4 * 128 * 2 - 16), L.LORA_ERR_ARG),       # over q
    (dict(workspace=None), L.LORA_ERR_ARG), (dict(workspace=P + 8), L.LORA_ERR_ARG), (dict(max_pages=1 << 28), L.LORA_ERR_SHAPE)])
def test_attention_weights_refuses(change, code):
    before = L.lora_launch_count()
    assert weigh(pages(), **change) == code
    assert L.lora_launch_count() == before


def test_attention_weights_without_tokens():
    before = L.lora_launch_count()
    assert weigh(pages(), T=0, weights=None, q=None, out=None, starts=None, lens=None, table=None, workspace=None) == L.LORA_OK
    assert L.lora_launch_count() == before
    assert L._lib.lora_tree_attention_weights_workspace_size(ctypes.byref(pages()), 4, 2, 2, -1) == 0


def test_attention_weights_workspace_sizes():
    """They grow with the table up to the widest that a call takes, and sizes that no call takes have none."""
    size = lambda *args: L._lib.lora_tree_attention_weights_workspace_size(ctypes.byref(pages()), *args)  # noqa: E731
    for S, T in ((1, 1), (128, 128), (1000, 4000)):
        sizes = [size(4, S, T, n) for n in (0, 1, 2, 4, 64, 8192, (1 << 27) - 65)]
        assert 0 < sizes[0] and sizes == sorted(sizes)
        kept = min(T, 16 * S // 2)                      # two query heads a kv head
        assert sizes[4] - sizes[0] == kept * 4 * 64 * 16 * 4
    assert size(4, 2, 2, (1 << 27) - 64) == 0 and size(4, 2, 1 << 29, 4) == 0
