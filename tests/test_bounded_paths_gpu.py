"""Sizes at which the kernels of a bounded cache take paths of their own: scores dropped from L2 once summed up, queries that
pass through the tensor cores' ring again for each key tile, moves of several rounds with many ranges.  Weights against their
definition in float64 on the device; bounds as in tests/test_weigh_gpu.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from segmented_gathered_rank_gb300 import inputs as I  # noqa: E402
from tests import decode_cases as C  # noqa: E402
from tests.test_decode_gpu import assert_within, cuda, host  # noqa: E402
from tests.test_evict_gpu import Eviction, random_scores, tied_scores  # noqa: E402
from tests.test_weigh_gpu import Weigh  # noqa: E402


def definition(w):
    """(weights, what was added, that with each term times its row's largest scale * sum |q k|) as [n_pages, n_kv, page]."""
    new, gain, loaded = (torch.zeros(w.weights.shape, dtype=torch.float64, device="cuda") for _ in range(3))
    new += cuda(w.weights).double()
    group = w.n_q // w.n_kv
    for s in range(w.S):
        b, n, length = int(w.starts[s]), int(w.starts[s + 1] - w.starts[s]), int(w.lens[s])
        if n == 0:
            continue
        ids = torch.from_numpy(w.table[s, : -(-length // w.page)].astype(np.int64)).cuda()
        tok = torch.arange(length, device="cuda")
        at = ids[tok // w.page] * w.page + tok % w.page                     # place in [n_pages * page]
        see = torch.ones(n, length, dtype=torch.bool, device="cuda")
        mask = torch.tril(torch.ones(n, n, dtype=torch.bool)) if w.masks is None else torch.from_numpy(w.masks[s])
        see[:, length - n:] = mask.cuda()
        for h in range(w.n_kv):
            k = w.kd[:, h].reshape(-1, w.d)[at].double()
            q = w.qd[b: b + n].view(n, w.n_q, w.d)[:, h * group: (h + 1) * group].double().reshape(n * group, w.d)
            on = see.repeat_interleave(group, 0)
            sc = (w.scale * (q @ k.T)).masked_fill(~on, -torch.inf)
            p = torch.softmax(sc, 1).masked_fill(~on, 0.0).nan_to_num(0.0)
            big = (w.scale * (q.abs() @ k.abs().T)).masked_fill(~on, 0.0).amax(1, keepdim=True)
            total, load = p.sum(0), (p * big).sum(0)
            for plane, value in ((gain, total), (loaded, load)):
                flat = plane[:, h].reshape(-1)
                flat[at] = value
                plane[:, h] = flat.view(-1, w.page)
            flat = new[:, h].reshape(-1)
            old = flat[at[: length - n]] * w.decay if w.decay else torch.zeros(length - n, dtype=torch.float64, device="cuda")
            flat[at] = total
            flat[at[: length - n]] += old
            new[:, h] = flat.view(-1, w.page)
    return new, gain, loaded


def check(w):
    torch.cuda.synchronize()
    assert int(w.status) == 0 and bool((w.ws[w.size:] == 0xAB).all())
    assert torch.equal(w.out, w.plain())
    ref, gain, loaded = definition(w)
    rows = int(np.diff(w.starts).max()) * (w.n_q // w.n_kv)
    bound = 2 * (w.d + 4) * C.U * loaded + (2.0 ** -17 + (rows + 2) * C.U) * gain + 4 * C.U * ref.abs() + 1e-30
    known = ~ref.isnan()
    assert torch.equal(w.wd.isnan(), ~known)                    # slots that hold no token
    off = (w.wd.double() - ref).abs()[known] / bound[known]
    assert float(off.max()) <= 1.0


# more tiles of 512 tokens than weigh_scores_kernel has blocks (seven a SM): 1152 and 1320
@pytest.mark.parametrize("dtype, requests, n_q, n_kv, d, page", [
    (I.BF16, [(1, 18000), (1, 18431), (1, 18432), (1, 17950)], 16, 8, 16, 64), (I.F32, [(1, 18000)] * 4, 8, 8, 16, 16),
    (I.BF16, [(2, 1030)] * 55, 16, 8, 64, 16), (I.BF16, [(3, 33000), (1, 900), (0, 40)], 40, 20, 8, 8)])
def test_scores_of_many_tiles(dtype, requests, n_q, n_kv, d, page):
    w = Weigh(41, dtype, requests, n_q, n_kv, d, page, decay=0.5).to_device()
    assert sum(n_kv * -(-length // 512) for n, length in requests if n) > 7 * torch.cuda.get_device_properties(0).multi_processor_count
    w.call()
    check(w)
    first = w.wd.clone()
    for _ in range(3):           # the workspace as the call before left it
        w.wd.copy_(cuda(w.weights))
        w.call()
        assert np.array_equal(host(w.wd), host(first), equal_nan=True)


# heads of 128 and tensor copies, more rows than the ring of query tiles holds (384): several key tiles a block, and few
@pytest.mark.parametrize("requests, n_q, n_kv, page, mask", [
    ([(100, 3000)] * 6, 16, 4, 16, None), ([(97, 700), (100, 130)], 8, 2, 16, "random"), ([(400, 900), (400, 2300), (1, 600)], 8, 2, 64, None),
    ([(110, 4000), (0, 5), (130, 2049), (64, 64)], 32, 8, 16, "tree"), ([(400, 400)], 32, 8, 256, None)])
def test_more_rows_than_the_ring_holds(requests, n_q, n_kv, page, mask):
    w = Weigh(42, I.BF16, requests, n_q, n_kv, 128, page, mask=mask, decay=0.9).to_device()
    w.call()
    check(w)


# ranges enough for rounds of 160 rows (heads of 128 bytes a slice), and of those several
@pytest.mark.parametrize("dtype, d, page", [(I.BF16, 128, 16), (I.BF16, 128, 1), (I.F32, 64, 16), (I.F32, 128, 8), (I.BF16, 192, 16)])
@pytest.mark.parametrize("S, n_kv", [(40, 2), (12, 8)])
def test_many_ranges_of_several_rounds(dtype, d, page, S, n_kv):
    rng = np.random.default_rng(S + d)
    lens = rng.integers(330, 1300, S)
    keep = np.minimum(lens - 1, rng.integers(161, 900, S))
    keep[::7] = (160, 161, 320, 480, 481, 641, 800)[: len(keep[::7])]
    keep[3] = -1
    for scores, weights in ((random_scores, "other"), (tied_scores, "same")):
        e = Eviction(S, dtype, lens, keep, 4, 33, n_kv, d, page, scores=scores, weights=weights).to_device()
        e.call()
        e.check()


# kept scores with many rows in one request and one in the others: places of the list by rows, tiles that begin in a block
@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("requests, n_q, n_kv, d, page", [
    ([(1, 1500)] * 10 + [(37, 1600)] + [(1, 700)] * 5, 8, 2, 64, 16), ([(190, 2600)] + [(1, 2048), (1, 300)] * 32, 8, 2, 128, 16),
    ([(0, 90), (17, 17), (1, 513), (33, 1025), (1, 5), (0, 3)] + [(1, 129)] * 12, 6, 2, 80, 8)])
def test_one_long_request_among_short_ones(dtype, requests, n_q, n_kv, d, page):
    w = Weigh(43, dtype, requests, n_q, n_kv, d, page, decay=0.9).to_device()
    assert w.T * (n_q // n_kv) <= 16 * w.S            # on average few rows, so that scores are kept
    w.call()
    check(w)
