"""Append with axes, attention that keeps weights and eviction together, as examples/bounded_cache.py runs them: every
call against its float64 definition on what the calls before it left, over images, decoded text and evictions."""
import importlib.util
import os

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
from tests.test_decode_gpu import CODE, TORCH, append_bound, assert_within, cuda, host  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_spec = importlib.util.spec_from_file_location("bounded_cache", os.path.join(ROOT, "examples", "bounded_cache.py"))
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("n_q, n_kv, d, page", [(8, 2, 64, 16), (6, 3, 80, 4), (4, 1, 128, 1)])
def test_stream_with_a_bounded_cache(dtype, n_q, n_kv, d, page):
    rng = np.random.default_rng(d + page)
    S, budget, slack, side, n_pos, rot = 3, 60, 6, 5, 400, d // 4 * 2
    longest = budget + slack + side * side + 8
    max_pages = -(-longest // page)
    n_pages = S * max_pages + 1
    table = rng.permutation(n_pages)[: S * max_pages].reshape(S, max_pages).astype(np.int32)
    kd, vd = (torch.full((n_pages, n_kv, page, d), float("nan"), dtype=TORCH[dtype], device="cuda") for _ in range(2))
    wd = torch.full((n_pages, n_kv, page), float("nan"), device="cuda")       # no slot is read before it is written
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = L.KvPages(CODE[dtype], kd, vd, n_pages, page, n_kv, d, status=status)
    axis = np.arange(rot // 2) % 3
    angle = np.arange(n_pos)[:, None] * 100.0 ** (-np.arange(rot // 2) * 2.0 / rot)
    cos_sin = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    norm = C.store(rng.normal(1, 0.1, d), dtype)
    decay, scale, first, recent = 0.75, float(np.float32(d ** -0.5)), 2, 7
    held, now = np.zeros(S, np.int64), np.zeros(S, np.int64)
    ws = torch.empty(max(L.lora_tree_attention_weights_workspace_size(kv, n_q, S, t, max_pages) for t in (S, S * side * side)),
                     dtype=torch.uint8, device="cuda")
    evictions = 0
    for step in range(26):
        # an image every eighth step for two of the requests, else one token each; the last request pauses now and then
        new, positions = [], []
        for s in range(S):
            n = side * side if step % 8 == 0 and s != 1 else 0 if s == 2 and step % 5 == 4 else 1
            new.append(n)
            positions.append(example.image(now[s], side) if n > 1 else np.full((n, 3), now[s]))
            now[s] += side if n > 1 else n
        positions, T = np.concatenate(positions).astype(np.int32), sum(new)
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        at = np.concatenate([h + np.arange(n) for h, n in zip(held, new)]).astype(np.int64)
        slots = table[np.repeat(np.arange(S), new), at // page].astype(np.int64) * page + at % page
        q, k, v = (C.store(rng.normal(0, 1, (T, h, d)), dtype) for h in (n_q, n_kv, n_kv))
        q_out = torch.empty(T, n_q * d, dtype=TORCH[dtype], device="cuda")
        k0, v0, w0 = host(kd), host(vd), host(wd)
        L.lora_kv_append_axes(kv, C.device(q.reshape(T, -1), dtype), C.device(k.reshape(T, -1), dtype), C.device(v.reshape(T, -1), dtype), T,
                              n_q, cuda(positions), 3, axis, cuda(slots), cuda(cos_sin), n_pos, rot, True, q_out,
                              q_norm=C.device(norm, dtype), k_norm=C.device(norm, dtype), eps=1e-6)
        ref = D.append_axes(q, k, v, positions, axis, slots, cos_sin, rot, True, norm, norm, float(np.float32(1e-6)), k0, v0)
        k1, v1 = host(kd), host(vd)
        assert_within(host(q_out).reshape(T, n_q, d), ref[0], append_bound(ref[0], dtype, d))
        written = ~np.isnan(ref[1])
        assert_within(k1[written], ref[1][written], append_bound(ref[1], dtype, d)[written])
        assert np.array_equal(np.isnan(k1), ~written) and np.array_equal(v1, ref[2], equal_nan=True)

        held += new
        lens = held.astype(np.int32)
        out = torch.empty_like(q_out)
        L.lora_tree_attention_weights(kv, wd, decay, q_out, n_q, cuda(starts), S, T, cuda(lens), cuda(table), max_pages, None, 0, scale, out, ws)
        c = C.Attention.__new__(C.Attention)
        c.d, c.dtype = d, dtype
        qh = host(q_out).reshape(T, n_q, d)
        o, mag, big = D.tree_attention(qh, k1, v1, starts, lens, table, None, scale)
        assert_within(host(out).reshape(T, n_q, d), o, c.bound(o, mag, big))
        w_ref, gain, loaded = D.attention_weights(qh, k1, starts, lens, table, None, scale, w0, decay)
        w1 = host(wd)
        known = ~np.isnan(w_ref)
        bound = 2 * (d + 4) * C.U * loaded + (2.0 ** -17 + (max(new) * n_q + 2) * C.U) * gain + 4 * C.U * np.abs(w_ref) + 1e-30
        assert np.array_equal(np.isnan(w1), ~known)
        assert_within(w1[known], w_ref[known], bound[known])

        keep = np.where(held > budget + slack, budget, -1).astype(np.int32)
        kept = torch.full((S, n_kv, budget), -7, dtype=torch.int32, device="cuda")
        new_lens = torch.empty(S, dtype=torch.int32, device="cuda")
        L.lora_kv_evict(kv, wd, wd, S, cuda(lens), cuda(table), max_pages, cuda(keep), first, recent, kept, budget, new_lens)
        planes, chosen, shorter = D.evict([k1, v1, w1], w1, lens, table, keep, first, recent)
        for got, want in zip((kd, vd, wd), planes):
            assert np.array_equal(host(got), want, equal_nan=True)
        for s, rows in enumerate(chosen):
            assert rows is None or np.array_equal(kept[s].cpu().numpy(), rows)
        evictions += sum(rows is not None for rows in chosen)
        held = new_lens.cpu().numpy().astype(np.int64)
        assert np.array_equal(held, shorter) and int(status) == 0
    assert evictions >= 4


def test_example_runs_and_stays_within_its_budget():
    torch.manual_seed(1)
    block = example.BoundedBlock(3, 64, 8, 36, recent=10, hidden=512, n_q=8, n_kv=2, head_dim=64, adapters=4, rank=8, max_position=512)
    adapter = torch.arange(3, device="cuda", dtype=torch.int32)
    now, cut = 0, 0
    for step in range(30):
        n = 36 if step % 10 == 0 else 1
        positions = example.image(now, 6) if n > 1 else np.full((1, 3), now)
        x = torch.randn(3 * n, 512, device="cuda").bfloat16()
        y = block.step(x, adapter.repeat_interleave(n), torch.from_numpy(np.tile(positions, (3, 1)).astype(np.int32)).cuda(),
                       **block.tables([n] * 3))
        assert bool(torch.isfinite(y.float()).all())
        block.held += n
        now += 6 if n > 1 else 1
        cut += block.evict()
        assert (block.held <= 64 + 8).all()
    assert cut >= 2 and int(block.status) == 0 and bool((block.weights >= 0).all())
    block.close()


class Step:
    """One step of all three calls on a cache of n_pages, whose pages `ids` hold the requests."""

    def __init__(self, n_pages, ids, S, seed, n_q=32, n_kv=8, d=128, page=16, length=700, budget=400):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.S, self.n_q, self.page, self.length, self.budget, self.max_pages = S, n_q, page, length, budget, -(-length // page)
        self.ids = ids
        self.planes = [torch.empty(n_pages, n_kv, page, d, **bf16), torch.empty(n_pages, n_kv, page, d, **bf16),
                       torch.empty(n_pages, n_kv, page, device="cuda")]
        for plane in self.planes:
            plane[ids] = torch.randn(len(ids), *plane.shape[1:], generator=g, device="cuda").to(plane.dtype).abs()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.kv = L.KvPages(L.LORA_BF16, *self.planes[:2], n_pages, page, n_kv, d, status=self.status)
        self.table = ids.int().view(S, self.max_pages).contiguous()
        last = length - 1
        self.slots = self.table[:, last // page].long() * page + last % page
        self.positions = torch.randint(0, 64, (S, 3), generator=g, device="cuda", dtype=torch.int32)
        self.cos_sin = torch.randn(64, d, generator=g, device="cuda")
        self.q, self.k, self.v = (torch.randn(S, h * d, generator=g, device="cuda").bfloat16() for h in (n_q, n_kv, n_kv))
        self.lens, self.keep = (torch.full((S,), x, dtype=torch.int32, device="cuda") for x in (length, budget))
        self.starts = torch.arange(S + 1, dtype=torch.int32, device="cuda")
        self.q_out, self.out = torch.empty_like(self.q), torch.empty_like(self.q)
        self.kept = torch.zeros(S, n_kv, budget, dtype=torch.int32, device="cuda")
        self.new_lens = torch.zeros_like(self.lens)
        self.ws = torch.empty(L.lora_tree_attention_weights_workspace_size(self.kv, n_q, S, S, self.max_pages), dtype=torch.uint8, device="cuda")
        self.axis = bytes(i % 3 for i in range(d // 2))

    def run(self, stream=None):
        L.lora_kv_append_axes(self.kv, self.q, self.k, self.v, self.S, self.n_q, self.positions, 3, self.axis, self.slots, self.cos_sin, 64,
                              self.k.shape[1] // self.kv.n_kv_heads, False, self.q_out, stream=stream)
        L.lora_tree_attention_weights(self.kv, self.planes[2], 0.5, self.q_out, self.n_q, self.starts, self.S, self.S, self.lens, self.table,
                                      self.max_pages, None, 0, 0.088, self.out, self.ws, stream=stream)
        L.lora_kv_evict(self.kv, self.planes[2], self.planes[2], self.S, self.lens, self.table, self.max_pages, self.keep, 2, 50, self.kept,
                        self.budget, self.new_lens, stream=stream)

    def results(self):
        torch.cuda.synchronize()
        assert int(self.status) == 0
        return [plane[self.ids] for plane in self.planes] + [self.q_out.clone(), self.out.clone(), self.kept.clone(), self.new_lens.clone()]


def test_pages_beyond_32_bits_of_elements():
    """The last pages of a cache of 2.7e9 elements give what the same pages of a small one do."""
    n = 165000
    assert n * 8 * 16 * 128 > 1 << 31
    ids = torch.randperm(2 * 44, generator=torch.Generator().manual_seed(3)).cuda()
    small, large = Step(2 * 44, ids, 2, 5), Step(n, n - 1 - ids, 2, 5)
    small.run()
    large.run()
    assert all(torch.equal(a, b) for a, b in zip(small.results(), large.results()))


def test_two_streams_at_once():
    """Calls on two streams with caches and workspaces of their own do not meet."""
    ids = torch.arange(16 * 44, device="cuda")
    alone = []
    for seed in (1, 2):
        step = Step(16 * 44, ids, 16, seed)
        step.run()
        alone.append(step.results())
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        steps = [Step(16 * 44, ids, 16, seed) for seed in (1, 2)]
        torch.cuda.synchronize()
        for step, stream in zip(steps, streams):
            step.run(stream)
        for step, want in zip(steps, alone):
            assert all(torch.equal(a, b) for a, b in zip(step.results(), want))


def test_a_captured_step_replays():
    ids = torch.arange(8 * 44, device="cuda")
    want = Step(8 * 44, ids, 8, 4)
    before = [p.clone() for p in want.planes]
    want.run()
    first = want.results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        want.run()
    for _ in range(3):
        for plane, old in zip(want.planes, before):
            plane.copy_(old)
        want.kept.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want.results(), first))
