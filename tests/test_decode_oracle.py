"""The decode-step definitions of oracle/decode.py against closed forms, brute force and torch (no GPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import decode as D
from tests import decode_cases as C


def test_w4_against_explicit_loops():
    x, codes, scales, zeros = C.w4_case(1, "f32", 3, 64, 5, 32, True)
    y, mag = D.w4_matvec(x, codes, scales, zeros, 32)
    for t in range(3):
        for n in range(5):
            terms = []
            for k in range(64):
                byte = int(codes[n, k // 2])
                code = byte & 15 if k % 2 == 0 else byte >> 4
                terms.append(float(x[t, k]) * float(scales[n, k // 32]) * (code - int(zeros[n, k // 32])))
            assert y[t, n] == pytest.approx(math.fsum(terms), rel=1e-12, abs=1e-12)
            assert mag[t, n] == pytest.approx(math.fsum(map(abs, terms)), rel=1e-12)


def test_w4_default_zero_is_eight():
    codes = np.full((2, 16), 0x88, np.uint8)
    y, _ = D.w4_matvec(np.ones((1, 32)), codes, np.ones((2, 1)), None, 32)
    assert np.array_equal(y, np.zeros((1, 2)))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product_and_keeps_lengths(interleaved):
    rng = np.random.default_rng(2)
    x, angle = rng.normal(size=(3, 12)), rng.normal(size=4)
    y = D.rotate(x, np.cos(angle), np.sin(angle), interleaved)
    a, b = (slice(0, 8, 2), slice(1, 8, 2)) if interleaved else (slice(0, 4), slice(4, 8))
    z = (x[:, a] + 1j * x[:, b]) * np.exp(1j * angle)
    assert np.allclose(y[:, a], z.real) and np.allclose(y[:, b], z.imag)
    assert np.array_equal(y[:, 8:], x[:, 8:])
    assert np.allclose(np.linalg.norm(y, axis=1), np.linalg.norm(x, axis=1))


def test_norm_of_constant_rows():
    assert np.allclose(D.rms_norm(np.full((1, 8), -3.0), np.full(8, 2.0), 0.0), -2.0)


def test_append_places_rows_and_leaves_the_rest():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(3, 4, 8)), rng.normal(size=(3, 2, 8)), rng.normal(size=(3, 2, 8))
    kp, vp = np.zeros((3, 2, 4, 8)), np.zeros((3, 2, 4, 8))
    q2, k2, v2 = D.append(q, k, v, [0, 0, 0], [5, -1, 11], np.zeros((1, 0)), 0, False, None, None, 1e-6, kp, vp)
    assert np.array_equal(q2, q)
    assert np.array_equal(k2[1, :, 1], k[0]) and np.array_equal(v2[2, :, 3], v[2])
    assert np.count_nonzero(k2) == 2 * 16 and np.count_nonzero(v2) == 2 * 16


def test_attention_matches_torch_softmax_on_a_dense_cache():
    c = C.Attention(4, "f32", [(3, 11)], 4, 2, 8, 16, mask="tree")
    out, mag, _ = D.tree_attention(c.q, c.k, c.v, c.starts, c.lens, c.table, c.masks, c.scale)
    k = torch.from_numpy(c.k[c.table[0, 0], :, :11]).double()
    v = torch.from_numpy(c.v[c.table[0, 0], :, :11]).double()
    q = torch.from_numpy(c.q).double()
    see = torch.ones(3, 11, dtype=torch.bool)
    see[:, 8:] = torch.from_numpy(c.masks[0])
    for h in range(4):
        s = (q[:, h] @ k[h // 2].T * c.scale).masked_fill(~see, -math.inf)
        p = torch.softmax(s, 1)
        assert np.allclose(out[:, h], (p @ v[h // 2]).numpy(), atol=1e-12)
        assert np.allclose(mag[:, h], (p @ v[h // 2].abs()).numpy(), atol=1e-12)


def test_attention_of_equal_keys_is_the_mean_of_visible_values():
    c = C.Attention(5, "f32", [(2, 6)], 1, 1, 8, 4)
    c.k[...] = np.where(np.isnan(c.k), np.nan, 1.0)
    out, _, _ = D.tree_attention(c.q, c.k, c.v, c.starts, c.lens, c.table, None, c.scale)
    v = c.v[c.table[0], 0].reshape(-1, 8)
    assert np.allclose(out[0, 0], v[:5].mean(0)) and np.allclose(out[1, 0], v[:6].mean(0))


def test_attention_rows_that_see_nothing_are_zero():
    c = C.Attention(6, "f32", [(3, 3), (0, 0), (1, 5)], 2, 1, 8, 4, mask=lambda rng, n: np.zeros((n, n), bool))
    out, _, _ = D.tree_attention(c.q, c.k, c.v, c.starts, c.lens, c.table, c.masks, c.scale)
    assert not out[:3].any() and out[3].any()


def test_mask_packing_round_trips():
    rng = np.random.default_rng(7)
    m = rng.random((70, 70)) < 0.5
    bits = C.pack_masks([m], 2)
    for i in (0, 31, 69):
        for j in (0, 1, 63, 64, 69):
            assert bool((int(bits[i, j // 64]) >> (j % 64)) & 1) == m[i, j]
