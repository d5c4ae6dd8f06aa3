"""lora_tree_attention_weights: scores are kept where the workspace holds them, else computed once more; either way out is
lora_tree_attention's and the weights are the definition's."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from segmented_gathered_rank_gb300 import inputs as I  # noqa: E402
from segmented_gathered_rank_gb300 import lora as L  # noqa: E402
from tests.test_weigh_gpu import Weigh  # noqa: E402

CASES = [   # requests, n_q, n_kv, d, page, mask
    ([(1, 777)], 32, 8, 128, 16, None), ([(1, 1), (1, 600), (0, 9), (1, 33)], 16, 4, 64, 16, None), ([(1, 300), (1, 31)], 7, 1, 80, 8, None),
    ([(1, 513)], 3, 3, 256, 64, None), ([(2, 100), (3, 290)], 4, 2, 128, 2, None), ([(4, 260), (1, 9), (3, 70)], 8, 2, 128, 16, "random"),
    ([(8, 500)], 4, 4, 24, 16, "tree"), ([(30, 300), (2, 50)], 8, 2, 64, 16, "tree")]


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in (c[0][0][0], c[0][0][1], len(c[0]), *c[1:])))
def test_a_workspace_without_room_for_scores(case, dtype):
    requests, n_q, n_kv, d, page, mask = case
    w = Weigh(31, dtype, requests, n_q, n_kv, d, page, mask=mask, decay=0.75).to_device()
    w.size = L.lora_tree_attention_weights_workspace_size(w.kv, n_q, w.S, w.T, 0)
    w.ws[w.size:] = 0xAB
    w.call()
    w.check()


@pytest.mark.parametrize("dtype", [I.BF16, I.F32])
@pytest.mark.parametrize("case", CASES[:4], ids=lambda c: "-".join(str(x) for x in (c[0][0][0], c[0][0][1], len(c[0]), *c[1:])))
def test_a_table_much_wider_than_what_is_cached(case, dtype):
    """By a workspace of what is cached, and by the table's own, whose scores lie far apart."""
    requests, n_q, n_kv, d, page, mask = case
    for own in (False, True):
        w = Weigh(32, dtype, requests, n_q, n_kv, d, page, mask=mask, decay=1.0)
        narrow = w.max_pages
        wide = np.full((w.S, 131072 // page), -1, np.int32)
        wide[:, :narrow] = w.table
        w.table, w.max_pages = wide, wide.shape[1]
        w.to_device()
        if not own:
            w.size = L.lora_tree_attention_weights_workspace_size(w.kv, n_q, w.S, w.T, narrow)
            w.ws[w.size:] = 0xAB
        w.call()
        w.check()


def test_a_workspace_that_holds_less_is_refused():
    for dtype in (I.BF16, I.F32):
        w = Weigh(33, dtype, [(1, 300)], 8, 2, 64, 16).to_device()
        least = L.lora_tree_attention_workspace_size(w.kv, 8, 1, 1)
        w.size = least - 16
        before = L.lora_launch_count()
        with pytest.raises(L.LoraError):
            w.call()
        assert L.lora_launch_count() == before
