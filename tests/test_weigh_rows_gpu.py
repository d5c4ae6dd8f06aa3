"""lora_tree_attention_weights: rows whose sum is not a number.  Such a row gives what it sees a weight that is none, by the
definition (oracle/decode.py), and what it does not see nothing.  Bounds as in tests/test_weigh_gpu.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from oracle import decode as D  # noqa: E402
from segmented_gathered_rank_gb300 import inputs as I  # noqa: E402
from tests import decode_cases as C  # noqa: E402
from tests.test_decode_gpu import assert_within, host  # noqa: E402
from tests.test_weigh_gpu import Weigh  # noqa: E402


def own_only(rng, n):
    """Each drafted token sees the prefix and itself."""
    return np.eye(n, dtype=bool)


def compare(w):
    """Against the definition, numbers that are none among them."""
    with np.errstate(invalid="ignore"):
        ref, gain, _ = D.attention_weights(w.q, w.k, w.starts, w.lens, w.table, w.masks, w.scale, w.weights, w.decay)
    # no row's largest scale * sum |q k| over its finite keys is above that of all rows and keys
    q, k = (np.where(np.isfinite(a), np.abs(a), 0.0).astype(np.float64) for a in (w.q, w.k))
    group = w.n_q // w.n_kv
    big = max(float((q[:, h * group: (h + 1) * group].reshape(-1, w.d) @ k[:, h].reshape(-1, w.d).T).max()) for h in range(w.n_kv)) * w.scale
    torch.cuda.synchronize()
    assert int(w.status) == 0
    got = host(w.wd)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    rows = int(np.diff(w.starts).max()) * group
    on = ~np.isnan(ref)
    bound = 2 * (w.d + 4) * C.U * big * gain + (2.0 ** -17 + (rows + 2) * C.U) * gain + 4 * C.U * np.abs(ref) + 1e-30
    assert_within(got[on], ref[on], bound[on])
    return ref


# bf16: warp MMAs with kept scores (up to 16 rows a kv head), tcgen05; fp32: few rows, tiles of rows with kept scores, without
@pytest.mark.parametrize("dtype, n, d", [(I.BF16, 3, 128), (I.BF16, 4, 80), (I.BF16, 40, 64), (I.F32, 2, 128), (I.F32, 20, 64),
                                         (I.F32, 70, 64)])
@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_a_drafted_key_that_is_not_finite_stays_with_the_row_that_sees_it(dtype, n, d, value):
    w = Weigh(21, dtype, [(n, n + 70), (n, n), (n, 2 * n + 5)], 8, 2, d, 16, mask=own_only, decay=1.0)
    c = int(w.lens[0]) - n + 1                    # drafted token 1 of the first request
    w.k[w.table[0, c // 16], :, c % 16] = value
    w.to_device().call()
    ref = compare(w)
    other = int(w.lens[0]) - n
    assert np.isnan(ref[w.table[0, c // 16], :, c % 16]).all() and np.isfinite(ref[w.table[0, other // 16], :, other % 16]).all()


@pytest.mark.parametrize("dtype, n, d", [(I.BF16, 3, 128), (I.BF16, 40, 64), (I.F32, 2, 80), (I.F32, 20, 64), (I.F32, 70, 64)])
def test_a_query_that_is_not_finite_stays_with_what_it_sees(dtype, n, d):
    w = Weigh(22, dtype, [(n, n + 70), (n, n + 3)], 8, 2, d, 16, mask=own_only, decay=0.5)
    w.q[0, 1] = np.nan                            # one head of one token of the first request
    w.to_device().call()
    ref = compare(w)
    assert np.isnan(ref).any() and np.isfinite(ref[w.table[1, 0], :, :2]).all()


@pytest.mark.parametrize("dtype, n", [(I.BF16, 2), (I.BF16, 40), (I.F32, 2), (I.F32, 20)])
def test_a_score_of_minus_infinity_beside_one_that_is_no_number(dtype, n):
    """Seen, it has no weight in a row of finite sum, and none that is a number in the other."""
    w = Weigh(23, dtype, [(n, n + 40)], 2, 2, 64, 16, mask=own_only, decay=1.0)
    w.q[:, :, 0] = C.store(np.abs(w.q[:, :, 0]) + np.float32(0.5), dtype)
    w.k[w.table[0, 0], :, 3, 0] = -np.inf         # a prefix token: minus infinity in every row
    c = int(w.lens[0]) - n + 1
    w.k[w.table[0, c // 16], :, c % 16] = np.nan
    w.to_device().call()
    compare(w)
