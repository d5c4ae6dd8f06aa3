"""A launch that fails is the failing call's error only: the next call, whose kernels run, does not report it again.  In a
process of its own, as the failure is a capture that is left by a call on the legacy stream."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import ctypes, glob, os, torch
from segmented_gathered_rank_gb300 import lora as L
torch.cuda.init()
names = ["libcudart.so.%d" % n for n in (13, 12)]
for name in names + sorted(glob.glob(os.path.join(os.path.dirname(torch.__file__), "..", "nvidia", "*", "lib", "libcudart.so.*"))):
    try:
        rt = ctypes.CDLL(name)
        break
    except OSError:
        pass
dev = dict(device="cuda")
k, v = (torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, **dev) for _ in range(2))
kv = L.KvPages(L.LORA_BF16, k, v, 4, 16, 1, 64)
scores, lens, keep, kept, new = torch.zeros(4, 1, 16, **dev), *(torch.full((n,), 8, dtype=torch.int32, **dev) for n in (1, 1, 8, 1))
table = torch.arange(4, dtype=torch.int32, **dev).view(1, 4)
x, slot = torch.ones(1, 64, dtype=torch.bfloat16, **dev), torch.zeros(1, dtype=torch.int64, **dev)
evict = lambda stream: L.lora_kv_evict(kv, scores, None, 1, lens, table, 4, keep, 0, 0, kept, 8, new, stream=stream)
evict(0)                # what the first call sets up is set up outside the capture
torch.cuda.synchronize()
side, graph = ctypes.c_void_p(), ctypes.c_void_p()
assert rt.cudaStreamCreate(ctypes.byref(side)) == 0 and rt.cudaStreamBeginCapture(side, 0) == 0
try:
    evict(0)            # the legacy stream would wait for the capture
    print("launched")
except L.LoraError as e:
    print("refused", e.status == L.LORA_ERR_CUDA)
rt.cudaStreamEndCapture(side, ctypes.byref(graph))
rt.cudaGetLastError()
L.lora_kv_append(kv, None, x, x, 1, 0, None, slot, None, 0, 0, False, None, stream=0)
torch.cuda.synchronize()
print("next", bool((k[0, 0, 0] == 1).all()))
"""


def test_the_next_call_does_not_report_a_launch_that_failed_before():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split("\n")[:2] == ["refused True", "next True"]
