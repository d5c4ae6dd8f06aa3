"""lora_kv_append_axes on the GPU against its float64 definition (oracle/decode.py).

Bound: the rounding of one store (bf16 2^-8 covers its half step twice over), and fewer than 2 log2(d) + 24 fp32
roundings, each of at most 2^-24 of the largest magnitude of a head (a rotation is at most sqrt(2) of it)."""
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
from tests.test_decode_gpu import CODE, TORCH, append_bound, append_case, assert_within, cuda, host  # noqa: E402


def sections(half, n):
    edge = np.round(np.cumsum([1] + [2] * (n - 1)) * half / (2 * n - 1))
    return np.searchsorted(edge, np.arange(half), side="right")


AXES = {"sections": sections, "cycle": lambda half, n: np.arange(half) % n,
        "last": lambda half, n: np.full(half, n - 1), "any": lambda half, n: np.random.default_rng(half).integers(0, n, half)}


class Axes:
    """A case of append_case with positions of several axes, and its device copies."""

    def __init__(self, case, dtype, n_axes, order, seed=0):
        self.case, self.dtype, self.n_axes = case, dtype, n_axes
        self.arrays = list(append_case(case, dtype, seed + case[0] + case[3]))
        rng = np.random.default_rng(seed + 17)
        self.arrays[6] = rng.integers(0, 97, (case[0], n_axes)).astype(np.int32)
        self.pair_axis = AXES[order](case[4] // 2, n_axes).astype(np.uint8)

    def reference(self):
        T, n_q, n_kv, d, rot, page, interleaved, norm, fused = self.case
        q, k, v, qn, kn, cos_sin, positions, slots, kp, vp = self.arrays
        return D.append_axes(q.reshape(T, n_q, d), k.reshape(T, n_kv, d), v.reshape(T, n_kv, d), positions, self.pair_axis, slots, cos_sin,
                             rot, interleaved, qn, kn, float(np.float32(1e-5)), kp, vp)

    def to_device(self, table_offset=0):
        T, n_q, n_kv, d, rot, page, interleaved, norm, fused = self.case
        q, k, v, qn, kn, cos_sin, positions, slots, kp, vp = self.arrays
        self.kd, self.vd = C.device(kp, self.dtype), C.device(vp, self.dtype)
        if fused:
            x = C.device(np.concatenate([q, k, v], 1), self.dtype)
            self.qkv = x[:, : n_q * d], x[:, n_q * d: (n_q + n_kv) * d], x[:, (n_q + n_kv) * d:]
        else:
            self.qkv = tuple(C.device(a, self.dtype) for a in (q, k, v))
        self.out = torch.full((T, n_q * d), float("nan"), dtype=TORCH[self.dtype], device="cuda")
        self.norms = tuple(None if a is None else C.device(a, self.dtype) for a in (qn, kn))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.kv = L.KvPages(CODE[self.dtype], self.kd, self.vd, len(kp), page, n_kv, d, status=self.status)
        flat = torch.empty(cos_sin.size + 4, device="cuda")[table_offset:][: cos_sin.size]      # an offset takes the table off 16 bytes
        self.table = flat.copy_(cuda(cos_sin).view(-1)).view(cos_sin.shape) if cos_sin.size else None
        self.positions, self.slots, self.n_pos = cuda(positions), cuda(slots), len(cos_sin)
        return self

    def call(self, stream=None, out=None):
        T, n_q, n_kv, d, rot, page, interleaved, norm, fused = self.case
        q, k, v = self.qkv
        L.lora_kv_append_axes(self.kv, q if n_q else None, k, v, T, n_q, self.positions if rot else None, self.n_axes,
                              self.pair_axis.tobytes(), self.slots, self.table, self.n_pos, rot, interleaved,
                              (self.out if out is None else out) if n_q else None, q_norm=self.norms[0], k_norm=self.norms[1], eps=1e-5,
                              stream=stream)

    def results(self):
        T, n_q, n_kv, d = self.case[:4]
        torch.cuda.synchronize()
        return host(self.out).reshape(T, n_q, d), host(self.kd), host(self.vd)

    def check(self):
        got, ref, d = self.results(), self.reference(), self.case[3]
        assert int(self.status) == 0
        assert_within(got[0], ref[0], append_bound(ref[0], self.dtype, d))
        assert_within(got[1], ref[1], append_bound(ref[1], self.dtype, d))
        assert np.array_equal(got[2], ref[2])
        page, slots, kp = self.case[5], self.arrays[7], self.arrays[8]
        written = np.zeros((len(kp), page), bool)
        for s in slots[slots >= 0]:
            written[s // page, s % page] = True
        keep = ~written[:, None, :, None] & np.ones_like(kp, bool)
        assert np.array_equal(got[1][keep], kp.astype(np.float64)[keep])     # slots that no token names are untouched


CASES = [   # T, n_q, n_kv, d, rot, page, interleaved, norm, fused
    (1, 32, 8, 128, 128, 16, False, True, True), (5, 4, 4, 64, 64, 1, True, False, True),
    (7, 7, 1, 80, 20, 8, False, True, False), (3, 2, 2, 8, 2, 4, False, True, False), (4, 2, 1, 8, 6, 4, True, True, True),
    (33, 16, 2, 256, 256, 64, False, True, True), (9, 6, 3, 112, 42, 32, False, True, True),
    (17, 8, 8, 96, 96, 128, False, False, False), (6, 0, 2, 128, 64, 16, False, True, False),
    (300, 28, 4, 128, 128, 16, True, True, True), (65, 40, 8, 192, 190, 1024, False, True, True),
    (2, 3, 1, 24, 0, 2, False, True, False), (1100, 8, 2, 64, 32, 16, False, False, True)]


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("n_axes, order", [(3, "sections"), (3, "cycle"), (4, "any"), (2, "last"), (1, "cycle")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_append_axes(case, n_axes, order, dtype):
    c = Axes(case, dtype, n_axes, order).to_device()
    c.call()
    c.check()


MANY = [   # enough bytes for the ring of whole tokens, in one type or both
    (700, 32, 8, 128, 128, 16, False, True, True), (800, 49, 7, 80, 24, 8, False, True, False), (900, 0, 32, 64, 64, 32, True, True, True),
    (500, 300, 100, 24, 8, 1, True, True, False), (1000, 20, 5, 256, 128, 64, False, False, True), (600, 30, 10, 192, 192, 4, True, True, False),
    (500, 900, 30, 8, 8, 16, False, True, True), (650, 48, 16, 112, 0, 16, False, True, True), (1300, 16, 8, 96, 48, 128, False, False, False)]


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("n_axes, order", [(3, "sections"), (4, "any"), (2, "last")])
@pytest.mark.parametrize("case", MANY, ids=lambda c: "-".join(map(str, c)))
def test_append_axes_of_many_tokens(case, n_axes, order, dtype):
    c = Axes(case, dtype, n_axes, order).to_device()
    c.call()
    c.check()
    again = Axes(case, dtype, n_axes, order).to_device()
    if not case[8] and case[1]:                 # queries in place
        again.out = again.qkv[0]
    again.call()
    assert all(np.array_equal(x, y) for x, y in zip(c.results(), again.results()))


def test_bad_positions_and_slots_of_many_tokens():
    c = Axes((1200, 32, 8, 64, 64, 8, False, True, True), I.BF16, 3, "last")
    n_pos, T = len(c.arrays[5]), 1200
    c.arrays[6][:, :2] = 1 << 30                # axes that no pair names
    c.arrays[6][17, 2], c.arrays[6][1100, 2] = -1, n_pos
    c.arrays[7][5], c.arrays[7][1199] = len(c.arrays[8]) * 8, 1 << 62
    c.to_device().call()
    got = c.results()
    assert int(c.status) == L.LORA_DEV_BAD_SLOT | L.LORA_DEV_BAD_POSITION
    c.arrays[6] = np.clip(c.arrays[6], 0, n_pos - 1)
    c.arrays[7][5] = c.arrays[7][1199] = -1
    ref = c.reference()
    assert_within(got[0], ref[0], append_bound(ref[0], I.BF16, 64))
    assert_within(got[1], ref[1], append_bound(ref[1], I.BF16, 64))
    assert np.array_equal(got[2], ref[2])


@pytest.mark.parametrize("interleaved", [False, True])
def test_table_off_16_bytes(interleaved):
    for T in (40, 1200):
        c = Axes((T, 32, 8, 64, 64, 16, interleaved, True, True), I.BF16, 3, "sections").to_device(table_offset=1)
        c.call()
        c.check()


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_equal_axes_are_plain_positions(dtype, interleaved):
    """A text token: every axis has its position, and the result is lora_kv_append's, bit for bit."""
    for case in [(37, 8, 2, 128, 128, 16, interleaved, True, True), (700, 32, 8, 128, 64, 16, interleaved, True, True)]:
        c = Axes(case, dtype, 3, "cycle")
        c.arrays[6][:] = c.arrays[6][:, :1]
        c.to_device().call()
        a = c.results()
        plain = torch.empty_like(c.out)
        L.lora_kv_append(c.kv, *c.qkv, case[0], case[1], c.positions[:, 0].contiguous(), c.slots, c.table, c.n_pos, case[4], interleaved,
                         plain, q_norm=c.norms[0], k_norm=c.norms[1], eps=1e-5)
        torch.cuda.synchronize()
        assert torch.equal(plain, c.out) and np.array_equal(host(c.kd), a[1])


def test_queries_in_place_and_no_tokens():
    c = Axes((50, 6, 2, 64, 48, 8, False, True, False), I.BF16, 3, "cycle").to_device()
    c.call()
    a = c.results()
    again = Axes((50, 6, 2, 64, 48, 8, False, True, False), I.BF16, 3, "cycle").to_device()
    again.out = again.qkv[0]
    again.call()
    b = again.results()
    assert all(np.array_equal(x, y) for x, y in zip(a, b))
    n = L.lora_launch_count()
    L.lora_kv_append_axes(c.kv, *c.qkv, 0, 6, c.positions, 3, c.pair_axis.tobytes(), c.slots, c.table, c.n_pos, 48, False, c.out)
    assert L.lora_launch_count() == n


def test_bad_positions_and_slots_are_flagged():
    c = Axes((4, 2, 1, 16, 8, 4, False, False, False), I.F32, 2, "cycle")
    n_pos = len(c.arrays[5])
    c.arrays[6] = np.array([[0, 1], [-5, 2], [3, n_pos], [4, 5]], np.int32)
    c.arrays[7] = np.array([0, 1, 2, len(c.arrays[8]) * 4], np.int64)
    c.to_device().call()
    got = c.results()
    assert int(c.status) == L.LORA_DEV_BAD_SLOT | L.LORA_DEV_BAD_POSITION
    c.arrays[6] = np.clip(c.arrays[6], 0, n_pos - 1)
    c.arrays[7][3] = -1
    ref = c.reference()
    assert_within(got[0], ref[0], append_bound(ref[0], I.F32, 16))
    assert_within(got[1], ref[1], append_bound(ref[1], I.F32, 16))


def test_an_axis_that_no_pair_names_is_not_looked_at():
    c = Axes((6, 2, 1, 32, 32, 4, False, True, False), I.BF16, 3, "last")
    c.arrays[6][:, :2] = 1 << 30
    c.to_device().call()
    c.arrays[6][:, :2] = 0
    c.check()


def test_streams_and_graphs():
    c = Axes((130, 16, 4, 128, 128, 16, False, True, True), I.BF16, 3, "sections").to_device()
    c.call()
    first = c.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.out.fill_(0)
    side.wait_stream(torch.cuda.current_stream())
    c.call(stream=side)
    side.synchronize()
    assert torch.equal(c.out, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    c.out.fill_(0)
    c.positions.add_(1).remainder_(97)
    graph.replay()
    c.arrays[6] = (c.arrays[6] + 1) % 97
    c.check()
