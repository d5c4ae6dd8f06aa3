"""lora_kv_evict on the GPU against its definition (oracle/decode.py).  Everything is moved or chosen: all equal."""
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
from tests.test_decode_gpu import CODE, cuda, host  # noqa: E402


def random_scores(rng, shape):
    return np.exp(2 * rng.normal(size=shape)).astype(np.float32)


def tied_scores(rng, shape):
    return rng.integers(0, 4, shape).astype(np.float32)


def odd_scores(rng, shape):
    f = rng.normal(size=shape).astype(np.float32)
    for value in (np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, np.float32(1e-45), np.finfo(np.float32).min, np.finfo(np.float32).max):
        f[rng.random(shape) < 0.08] = value
    return f


def near_scores(rng, shape):
    """Apart in their last bits only."""
    return (np.float32(1.0) + rng.integers(0, 64, shape) * np.finfo(np.float32).eps).astype(np.float32)


class Eviction:
    def __init__(self, seed, dtype, lens, keep, first, recent, n_kv, d, page, scores=random_scores, weights="other", ld=None, max_pages=None):
        rng = np.random.default_rng(seed)
        self.S, self.dtype, self.n_kv, self.d, self.page, self.first, self.recent = len(lens), dtype, n_kv, d, page, first, recent
        self.lens, self.keep = np.array(lens, np.int32), np.broadcast_to(np.array(keep, np.int32), len(lens)).copy()
        used = [-(-int(n) // page) for n in self.lens]
        self.max_pages, self.n_pages = max(1, max(used)) if max_pages is None else max_pages, sum(used) + 2
        ids = rng.permutation(self.n_pages)
        self.table = np.full((self.S, self.max_pages), -1, np.int32)
        at = 0
        for s, n in enumerate(used):
            self.table[s, :n] = ids[at: at + n]
            at += n
        shape = (self.n_pages, n_kv, page)
        self.k, self.v = (C.store(rng.normal(size=(*shape, d)).astype(np.float32), dtype) for _ in range(2))
        self.scores = scores(rng, shape)
        self.weights = {"other": random_scores(rng, shape), "same": self.scores, None: None}[weights]
        self.mode, self.ld = weights, max(1, int(self.keep.max())) if ld is None else ld

    def to_device(self):
        self.kd, self.vd = C.device(self.k, self.dtype), C.device(self.v, self.dtype)
        self.sd = cuda(self.scores)
        self.wd = {"other": lambda: cuda(self.weights), "same": lambda: self.sd, None: lambda: None}[self.mode]()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.kv = L.KvPages(CODE[self.dtype], self.kd, self.vd, self.n_pages, self.page, self.n_kv, self.d, status=self.status)
        self.tables = [cuda(a) for a in (self.lens, self.table, self.keep)]
        self.kept = torch.full((self.S, self.n_kv, self.ld), -7, dtype=torch.int32, device="cuda")
        self.new_lens = torch.full((self.S + 1,), -7, dtype=torch.int32, device="cuda")
        return self

    def call(self, stream=None):
        lens, table, keep = self.tables
        L.lora_kv_evict(self.kv, self.sd, self.wd, self.S, lens, table, self.max_pages, keep, self.first, self.recent,
                        self.kept if self.ld else None, self.ld, self.new_lens, stream=stream)

    def check(self, status=0, lens=None, keep=None):
        torch.cuda.synchronize()
        planes = [self.k, self.v] + ([] if self.weights is None else [self.weights])
        lens = self.lens if lens is None else lens
        ref, kept, new_lens = D.evict(planes, self.scores, lens, self.table, self.keep if keep is None else keep, self.first, self.recent)
        assert int(self.status) == status
        assert np.array_equal(self.new_lens[:-1].cpu().numpy(), np.where(np.array(lens) == self.lens, new_lens, self.lens))
        assert int(self.new_lens[-1]) == -7
        want = np.full((self.S, self.n_kv, self.ld), -7)
        for s, rows in enumerate(kept):
            if rows is not None:
                want[s, :, : rows.shape[1]] = rows
        assert np.array_equal(self.kept.cpu().numpy(), want)
        got = [host(self.kd), host(self.vd)] + ([] if self.wd is None else [host(self.wd)])
        for g, r in zip(got, ref):
            assert np.array_equal(g, np.asarray(r, np.float64), equal_nan=True)
        if self.mode != "same":
            assert np.array_equal(self.sd.cpu().numpy(), self.scores, equal_nan=True)      # read only


CASES = [   # lens, keep, first, recent, n_kv, d, page
    ([1], 0, 0, 0, 1, 8, 1), ([2], 1, 0, 0, 2, 64, 16), ([2], 1, 5, 5, 2, 64, 16), ([33], 32, 4, 8, 2, 128, 8),
    ([40, 0, 17, 5], [10, 3, 16, 5], 2, 3, 3, 80, 8), ([300, 299, 301, 1, 64], [64, 298, -1, 0, 64], 1, 0, 2, 128, 16),
    ([700], 699, 0, 0, 1, 256, 64), ([1000], 37, 0, 37, 2, 64, 32), ([1000], 37, 40, 0, 2, 64, 32), ([1000], 37, 30, 30, 2, 24, 1024),
    ([513, 1025], [512, 511], 16, 64, 8, 128, 16), ([5000], 1234, 7, 100, 4, 112, 4), ([640] * 40, [13 * i for i in range(40)], 3, 9, 5, 16, 2),
    ([4200] * 3, 4096, 4, 128, 2, 128, 128)]


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("scores", [random_scores, tied_scores, odd_scores, near_scores], ids=lambda f: f.__name__.split("_")[0])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in (c[0][0], len(c[0]), *c[2:])))
def test_evict(case, scores, dtype):
    for weights in ("other", "same", None):
        e = Eviction(len(case[0]) + case[5], dtype, *case, scores=scores, weights=weights).to_device()
        e.call()
        e.check()


def test_all_scores_equal():
    """Ties: the lower indices stay."""
    e = Eviction(1, I.BF16, [777], [300], 0, 10, 2, 64, 16, scores=lambda rng, shape: np.full(shape, 0.25, np.float32)).to_device()
    e.call()
    e.check()
    assert np.array_equal(e.kept[0, 0].cpu().numpy(), np.concatenate([np.arange(290), np.arange(767, 777)]))


@pytest.mark.parametrize("lens, keep, n_kv, d, page", [([140001], [3001], 1, 8, 64), ([140001], [139000], 1, 8, 16),
                                                       ([40000] + [50] * 200, [20001] + [49] * 200, 2, 8, 16)])
def test_more_tokens_than_shared_memory_holds(lens, keep, n_kv, d, page):
    for scores in (random_scores, tied_scores):
        e = Eviction(9, I.BF16, lens, keep, 4, 50, n_kv, d, page, scores=scores, weights="same").to_device()
        e.call()
        e.check()


def test_evicted_again_and_again():
    """Budget by budget: what one call leaves is the next one's input."""
    e = Eviction(3, I.BF16, [900, 400], [700, 399], 4, 32, 2, 64, 16, weights="same").to_device()
    for budget in (700, 699, 350, 64, 1):
        e.tables[2].fill_(budget)
        e.keep[:] = budget
        e.call()
        e.check()
        e.k, e.v = (host(t).astype(np.float32) for t in (e.kd, e.vd))
        e.scores = e.weights = e.sd.cpu().numpy()
        e.lens = e.new_lens[:-1].cpu().numpy()
        e.tables[0].copy_(e.new_lens[:-1])
        e.kept.fill_(-7)


@pytest.mark.parametrize("what", ["length", "negative", "budget", "page", "page_low"])
def test_bad_tables_leave_the_request_as_it_is(what):
    e = Eviction(5, I.BF16, [200, 100, 150], [50, 40, 30], 2, 5, 2, 64, 8, ld=50)
    lens, keep, status = e.lens.copy(), e.keep.copy(), L.LORA_DEV_BAD_LENGTH
    if what == "length":
        e.lens[1] = e.max_pages * e.page + 1
    elif what == "negative":
        e.lens[1] = -3
    elif what == "budget":
        e.keep[1] = 51
    else:
        e.table[1, 3] = e.n_pages if what == "page" else -1
        status = L.LORA_DEV_BAD_PAGE
    e.to_device().call()
    keep[1] = -1            # as if it were not to be touched
    e.check(status, lens=lens if what in ("length", "negative") else None, keep=keep)


def test_no_budget_to_keep_and_no_room_for_indices():
    e = Eviction(6, I.F32, [30, 8], [0, 0], 2, 2, 2, 16, 4, ld=0).to_device()
    e.call()
    torch.cuda.synchronize()
    assert e.new_lens.tolist() == [0, 0, -7] and int(e.status) == 0
    assert np.array_equal(host(e.kd), e.k.astype(np.float64))


def test_shared_prefix_pages_that_all_keep_are_not_written():
    """The first tokens stay where they are, so requests may share the pages that hold nothing else."""
    e = Eviction(7, I.BF16, [100, 120], [40, 50], 16, 4, 2, 64, 8)
    e.table[1, :2] = e.table[0, :2]
    e.to_device().call()
    e.check()


def test_streams_graphs_and_repeats():
    e = Eviction(8, I.BF16, [3000, 2000, 2500], [1024, 1024, 1024], 4, 64, 4, 128, 16).to_device()
    e.call()
    e.check()
    first = [t.clone() for t in (e.kd, e.vd, e.wd, e.kept, e.new_lens)]
    for _ in range(5):
        f = Eviction(8, I.BF16, [3000, 2000, 2500], [1024, 1024, 1024], 4, 64, 4, 128, 16).to_device()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        f.call(stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (f.kd, f.vd, f.wd, f.kept, f.new_lens)))
    g = Eviction(8, I.BF16, [3000, 2000, 2500], [1024, 1024, 1024], 4, 64, 4, 128, 16).to_device()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.call()
    g.tables[0][1] = 700             # another batch in the same buffers
    g.lens[1] = 700
    g.tables[2][2] = 77
    g.keep[2] = 77
    graph.replay()
    g.check()


@pytest.mark.parametrize("weights", ["other", None])
@pytest.mark.parametrize("S", [18, 19, 37, 38, 39, 50, 51, 75, 76, 77, 152, 153, 305, 609])
def test_as_many_ranges_as_there_are_blocks(S, weights):
    """Around the sizes at which ranges are halved, dealt out or run by longer rounds (two kv heads of 128 bytes)."""
    rng = np.random.default_rng(S)
    e = Eviction(S, I.BF16, rng.integers(0, 90, S), rng.integers(-1, 60, S), 2, 5, 2, 64, 8, weights=weights).to_device()
    e.call()
    e.check()
