"""lora_tree_attention_weights on the GPU against its float64 definition (oracle/decode.py).

out is lora_tree_attention's, bit for bit.  A weight is a sum of probabilities 2^(s - lse).  A score s is off by at
most (d + 4) u of scale * sum |q k| (u = 2^-24; tests/decode_cases.py), lse by as much and by the exponentials' and
sums' 2^-18; the exponent's own rounding (|s - lse| up to some hundreds times u) and the last exponential's make it
2^-17 in all, and a sum over r rows rounds at most r + 2 times.  Nothing is rounded to bf16 on the way."""
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
from tests.test_decode_gpu import CODE, TORCH, assert_within, cuda, host  # noqa: E402


class Weigh(C.Attention):
    """An attention case with weights that earlier steps left (NaN where nothing has been)."""

    def __init__(self, *args, decay=1.0, stale=np.nan, **kw):
        super().__init__(*args, **kw)
        rng = np.random.default_rng(self.T + self.S)
        self.decay = float(np.float32(decay))
        self.weights = np.full(self.k.shape[:3], stale, np.float32)
        for s in range(self.S):
            prefix = int(self.lens[s]) - int(self.starts[s + 1] - self.starts[s])
            for c in range(prefix if decay else 0):
                self.weights[self.table[s, c // self.page], :, c % self.page] = np.exp(rng.normal(size=self.n_kv)) / self.lens[s]

    def to_device(self):
        self.kd, self.vd, self.qd = C.device(self.k, self.dtype), C.device(self.v, self.dtype), C.device(self.q.reshape(self.T, -1), self.dtype)
        self.wd = cuda(self.weights)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.kv = L.KvPages(CODE[self.dtype], self.kd, self.vd, self.n_pages, self.page, self.n_kv, self.d, status=self.status)
        self.tables = [cuda(a) for a in (self.starts, self.lens, self.table)]
        self.bits_d = cuda(self.bits)
        self.out = torch.full((self.T, self.n_q * self.d), 7.0, dtype=TORCH[self.dtype], device="cuda")
        size = L.lora_tree_attention_weights_workspace_size(self.kv, self.n_q, self.S, self.T, self.max_pages)
        self.ws = torch.full((size + 256,), 0xAB, dtype=torch.uint8, device="cuda")
        self.size = size
        return self

    def call(self, stream=None):
        starts, lens, table = self.tables
        L.lora_tree_attention_weights(self.kv, self.wd, self.decay, self.qd, self.n_q, starts, self.S, self.T, lens, table, self.max_pages,
                                      self.bits_d, self.words, self.scale, self.out, self.ws, ws_bytes=self.size, stream=stream)

    def plain(self):
        starts, lens, table = self.tables
        out = torch.full_like(self.out, 7.0)
        ws = torch.empty(L.lora_tree_attention_workspace_size(self.kv, self.n_q, self.S, self.T), dtype=torch.uint8, device="cuda")
        L.lora_tree_attention(self.kv, self.qd, self.n_q, starts, self.S, self.T, lens, table, self.max_pages, self.bits_d, self.words,
                              self.scale, out, ws)
        return out

    def check(self):
        torch.cuda.synchronize()
        assert int(self.status) == 0
        assert bool((self.ws[self.size:] == 0xAB).all())
        assert torch.equal(self.out, self.plain())
        ref, gain, loaded = D.attention_weights(self.q, self.k, self.starts, self.lens, self.table, self.masks, self.scale, self.weights,
                                                self.decay)
        got = host(self.wd)
        written = np.zeros(self.weights.shape, bool)
        rows = 1
        for s in range(self.S):
            n = int(self.starts[s + 1] - self.starts[s])
            rows = max(rows, n * (self.n_q // self.n_kv))
            for c in range(int(self.lens[s]) if n else 0):
                written[self.table[s, c // self.page], :, c % self.page] = True
        assert np.array_equal(self.wd.cpu().numpy()[~written], self.weights[~written], equal_nan=True)     # as they were
        bound = 2 * (self.d + 4) * C.U * loaded + (2.0 ** -17 + (rows + 2) * C.U) * gain + 4 * C.U * np.abs(ref) + 1e-30
        assert_within(got[written], ref[written], bound[written])


CASES = [   # requests (drafted, cached), n_q, n_kv, d, page, mask, decay
    ([(1, 1)], 8, 2, 64, 16, None, 1.0), ([(1, 777)], 32, 8, 128, 16, None, 1.0), ([(1, 2)], 4, 4, 128, 1, None, 0.5),
    ([(1, 100), (1, 1), (0, 50), (1, 3000), (1, 64)], 16, 4, 128, 16, None, 0.98), ([(1, 300), (1, 31)], 7, 1, 80, 8, None, 1.0),
    ([(1, 5000)], 8, 1, 64, 32, None, 0.0), ([(1, 513), (1, 1025), (1, 40)], 3, 3, 256, 64, None, 0.25),
    ([(1, 130)] * 70, 4, 2, 64, 2, None, 0.9), ([(3, 200), (0, 0), (5, 5), (2, 1000)], 6, 2, 112, 4, "tree", 1.0),
    ([(4, 260), (1, 9), (7, 70)], 8, 2, 128, 16, "random", 0.5), ([(16, 900)], 8, 8, 64, 16, "tree", 1.0),
    ([(33, 700), (20, 1500), (0, 10), (64, 64)], 16, 4, 128, 64, "tree", 1.0), ([(64, 3000)], 32, 8, 128, 16, None, 0.0),
    ([(100, 400), (3, 90)], 8, 1, 64, 8, "random", 0.7), ([(129, 200)], 4, 2, 128, 16, None, 1.0), ([(200, 1200), (90, 900)], 2, 1, 64, 128, None, 0.9),
    ([(40, 333)], 6, 3, 80, 16, "tree", 1.0), ([(50, 600), (60, 61)], 4, 1, 256, 1, "tree", 0.5), ([(70, 500)], 4, 4, 192, 32, None, 0.3),
    ([(30, 260), (11, 400)], 14, 2, 128, 4, "random", 1.0), ([(70, 300)], 12, 3, 80, 16, "tree", 0.8),
    ([(90, 91), (150, 500)], 6, 2, 112, 2, None, 1.0), ([(65, 129)], 32, 8, 24, 8, "random", 0.0)]


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in (c[0][0][0], c[0][0][1], len(c[0]), *c[1:])))
def test_weights(case, dtype):
    requests, n_q, n_kv, d, page, mask, decay = case
    w = Weigh(50 + d, dtype, requests, n_q, n_kv, d, page, mask=mask, decay=decay).to_device()
    w.call()
    w.check()


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("n, d", [(2, 128), (12, 80), (40, 64), (40, 128)])
def test_rows_that_see_nothing_and_wide_scores(dtype, n, d):
    """Mask rows of zeros with no context, and scores far apart (most probabilities are 0)."""
    w = Weigh(3, dtype, [(n, n), (n, 200)], 8, 2, d, 16, mask=lambda rng, n: rng.random((n, n)) < 0.2, decay=1.0, scale=1.5).to_device()
    w.call()
    w.check()
    none = Weigh(4, dtype, [(n, n), (n, 2 * n)], 8, 2, d, 16, mask=lambda rng, n: np.zeros((n, n), bool), decay=1.0).to_device()
    none.call()
    none.check()
    assert bool((none.out[:n] == 0).all())


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("n, d", [(1, 128), (3, 80), (40, 128)])
def test_masked_keys_that_are_not_finite(dtype, n, d):
    w = Weigh(6, dtype, [(n, 100), (n, 3 * n + 40)], 4, 2, d, 16, mask=lambda rng, n: np.tril(np.ones((n, n), bool), -1), decay=0.5)
    for s in range(2):       # the last drafted token of each request, which nobody sees
        c = int(w.lens[s]) - 1
        w.k[w.table[s, c // 16], :, c % 16] = (np.nan, np.inf)[s]
    clean = Weigh(6, dtype, [(n, 100), (n, 3 * n + 40)], 4, 2, d, 16, mask=lambda rng, n: np.tril(np.ones((n, n), bool), -1), decay=0.5)
    w.to_device().call()
    clean.to_device().call()
    torch.cuda.synchronize()
    assert torch.equal(w.out, clean.out)
    for s in range(2):
        c = int(w.lens[s]) - 1
        assert bool((w.wd[w.table[s, c // 16], :, c % 16] == 0).all())
    assert np.array_equal(host(w.wd), host(clean.wd), equal_nan=True)


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("requests", [[(1, 2500), (1, 70), (1, 900)], [(5, 1500), (9, 300)], [(48, 2000), (64, 700)]])
def test_repeats_streams_and_graphs(dtype, requests):
    make = lambda: Weigh(8, dtype, requests, 16, 4, 128, 16, decay=0.9).to_device()  # noqa: E731
    a = make()
    a.call()
    a.check()
    for _ in range(5):
        b = make()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        b.call(stream=side)
        side.synchronize()
        assert np.array_equal(host(a.wd), host(b.wd), equal_nan=True) and torch.equal(a.out, b.out)
    g = make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.call()
    graph.replay()
    g.check()
    before = g.wd.clone()
    graph.replay()                       # the next step: what the first left is read
    torch.cuda.synchronize()
    prefix = g.lens - np.diff(g.starts)
    for s in range(g.S):
        for c in (0, int(prefix[s]) - 1):
            at = g.table[s, c // 16], slice(None), c % 16
            first = host(before[at]) - g.decay * g.weights[at]
            assert np.allclose(host(g.wd[at]), g.decay * host(before[at]) + first, rtol=1e-5, atol=1e-9)


def test_weights_of_a_page_outside_the_cache():
    """The page is flagged and clamped as in the attention; no weight is written for it."""
    for dtype, n in ((I.BF16, 1), (I.BF16, 40), (I.F32, 1), (I.F32, 12)):
        w = Weigh(9, dtype, [(n, 200)], 8, 2, 128, 16, decay=1.0, garbage=0.5, stale=0.0)
        w.table[0, 2] = w.n_pages
        w.to_device().call()
        torch.cuda.synchronize()
        assert int(w.status) == L.LORA_DEV_BAD_PAGE
        used = [int(x) for i, x in enumerate(w.table[0]) if i != 2]
        other = [i for i in range(w.n_pages) if i not in used]
        assert np.array_equal(w.wd.cpu().numpy()[other], w.weights[other])
        assert bool(torch.isfinite(w.wd).all())


def test_bad_segments_and_lengths_stay_inside():
    for dtype in (I.BF16, I.F32):
        w = Weigh(10, dtype, [(2, 50), (3, 60)], 4, 2, 64, 8, decay=1.0, garbage=0.25, stale=0.0)
        w.lens[0] = w.max_pages * 8 + 100                       # clamped to the table, whose missing pages are clamped too
        w.starts[2] = 4
        w.to_device().call()
        torch.cuda.synchronize()
        assert int(w.status) & (L.LORA_DEV_BAD_LENGTH | L.LORA_DEV_BAD_SEGMENTS)
        assert bool((w.ws[w.size:] == 0xAB).all()) and bool(torch.isfinite(w.wd).all())


@pytest.mark.parametrize("dtype, T, S, d", [(I.BF16, 32, 64, 64), (I.BF16, 512, 16, 64), (I.F32, 32, 64, 128), (I.F32, 512, 16, 64)])
def test_overlapping_segments_leave_the_weights(dtype, T, S, d):
    k, v = (torch.randn(4, 1, 64, d, device="cuda").to(TORCH[dtype]) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = L.KvPages(CODE[dtype], k, v, 4, 64, 1, d, status=status)
    q = torch.randn(T, 8 * d, device="cuda").to(TORCH[dtype])
    out, weights = torch.full_like(q, float("nan")), torch.full((4, 1, 64), 5.0, device="cuda")
    starts = torch.tensor([0, T] * (S // 2) + [0], dtype=torch.int32, device="cuda")
    lens, table = torch.full((S,), 512, dtype=torch.int32, device="cuda"), torch.zeros((S, 8), dtype=torch.int32, device="cuda")
    ws = torch.empty(L.lora_tree_attention_weights_workspace_size(kv, 8, S, T, 8), dtype=torch.uint8, device="cuda")
    L.lora_tree_attention_weights(kv, weights, 1.0, q, 8, starts, S, T, lens, table, 8, None, 0, 0.1, out, ws)
    torch.cuda.synchronize()
    assert int(status) == L.LORA_DEV_BAD_SEGMENTS and bool(torch.isnan(out).all()) and bool((weights == 5).all())


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("d", [64, 80, 128])
def test_workspace_of_the_largest_call_serves_every_smaller_one(dtype, d):
    k, v = (torch.randn(40, 2, 16, d, device="cuda").to(TORCH[dtype]) for _ in range(2))
    kv = L.KvPages(CODE[dtype], k, v, 40, 16, 2, d)
    for group in (1, 4, 16):
        most = L.lora_tree_attention_weights_workspace_size(kv, 2 * group, 128, 128, 40)
        for T in (1, 2, 7, 16, 33, 64, 127, 128):
            for S in {1, 2, (T + 15) // 16, (T + 1) // 2, T, 128}:
                for pages in (1, 9, 40):
                    assert 0 < L.lora_tree_attention_weights_workspace_size(kv, 2 * group, S, T, pages) <= most


def test_no_tokens():
    w = Weigh(11, I.BF16, [(1, 30)], 4, 2, 64, 8).to_device()
    n = L.lora_launch_count()
    L.lora_tree_attention_weights(w.kv, w.wd, 1.0, w.qd, 4, w.tables[0], 1, 0, w.tables[1], w.tables[2], w.max_pages, None, 0, 0.1, w.out, w.ws)
    assert L.lora_launch_count() == n
    assert np.array_equal(w.wd.cpu().numpy(), w.weights, equal_nan=True)
