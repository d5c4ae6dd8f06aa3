"""Decode-step operators on the GPU where units, tables and sizes meet (definitions: oracle/decode.py; bounds:
tests/decode_cases.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from segmented_gathered_rank_gb300 import inputs as I  # noqa: E402
from tests import decode_cases as C  # noqa: E402
from tests.test_decode_gpu import check_attention, run_attention  # noqa: E402


# ----------------------------------------------------------------------------
# tcgen05 attention: units in which only one softmax stream has a part, in turn with units in which both have
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("requests", [
    [(16, 30 + i) if i % 2 else (16, 700 + 40 * (i % 7)) for i in range(100)],     # one key tile, then several: 64 rows a unit
    [(9, 9 + i % 90) if i % 4 else (25, 1500) for i in range(140)],                # three units of one tile in a row
    [(6, 90 + i) if i % 2 else (70, 300 + i) for i in range(100)],                 # 24 rows a unit, then 256 and 24
], ids=["one_tile", "one_tile_runs", "few_rows"])
def test_attention_streams_take_turns(requests, d):
    c = C.Attention(400 + d, I.BF16, requests, 16, 4, d, 16, mask="tree")
    got = check_attention(c)
    for _ in range(10):
        assert np.array_equal(run_attention(c), got)
