"""The decode-step operators together, as examples/decode_attention.py runs them, against their definitions in float64
with the block's own roundings to bf16 in between."""
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
from tests.parity import TOL_Y, rel_err  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_spec = importlib.util.spec_from_file_location("decode_attention", os.path.join(ROOT, "examples", "decode_attention.py"))
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


def host(t):
    return t.detach().float().cpu().numpy()


def bf16(a):
    return I.round_to_bf16(np.asarray(a, np.float32))


@pytest.mark.parametrize("requests,drafts,context", [(5, 1, 70), (3, 7, 200), (2, 40, 90)])
def test_decode_step(requests, drafts, context):
    torch.manual_seed(requests)
    block = example.AttentionBlock(hidden=512, n_q=8, n_kv=2, head_dim=64, adapters=4, rank=8, page=16, n_pages=64, max_tokens=128,
                                   max_position=1024, seed=requests)
    t = example.batch(block, requests, drafts, context, adapters=4, seed=drafts)
    T = requests * drafts
    x = torch.randn(T, 512, device="cuda").bfloat16()
    k0, v0 = host(block.k_pages), host(block.v_pages)
    y = block.step(x, **t)
    again = y.clone()
    block.k_pages.copy_(torch.from_numpy(k0))
    block.v_pages.copy_(torch.from_numpy(v0))
    assert torch.equal(block.step(x, **t), again) and int(block.status) == 0

    adapter = host(t["token_adapter"]).astype(np.int32)

    def project(name, a):
        p = block.proj[name]
        base, _ = D.w4_matvec(a, p.codes_host, p.scales_host, p.zeros_host, p.group)
        delta = np.zeros_like(base)
        for i, ad in enumerate(adapter):
            at, b = block.adapters_host[p.index, int(ad)]
            delta[i] = (a[i].astype(np.float64) @ at.T.astype(np.float64)) @ b.astype(np.float64)
        return bf16(bf16(base) + delta)

    xh = host(x)
    q, k, v = project("q", xh), project("k", xh), project("v", xh)
    q2, kp, vp = D.append(q.reshape(T, 8, 64).astype(np.float64), k.reshape(T, 2, 64).astype(np.float64), v.reshape(T, 2, 64),
                          host(t["positions"]).astype(int), t["slots"].cpu().numpy(), host(block.cos_sin), 64, False, host(block.q_norm),
                          host(block.k_norm), 1e-6, k0, v0)
    bits = t["tree_mask"].cpu().numpy()[:, 0]
    masks = [np.array([[(int(bits[s * drafts + i]) >> j) & 1 for j in range(drafts)] for i in range(drafts)], bool) for s in range(requests)]
    out, _, _ = D.tree_attention(bf16(q2), bf16(kp), vp, t["starts"].cpu().numpy(), t["lens"].cpu().numpy(), t["table"].cpu().numpy(), masks, 0.125)
    ref = project("o", bf16(out.reshape(T, -1)))
    assert rel_err(host(again), ref) <= TOL_Y[I.BF16]
    block.close()


def test_workspace_size_serves_smaller_batches():
    block = example.AttentionBlock(hidden=512, n_q=8, n_kv=2, head_dim=64, adapters=1, rank=8, n_pages=8, max_tokens=16, max_position=64)
    assert all(L.lora_tree_attention_workspace_size(block.kv, 8, s, 16) <= block.workspace.numel() for s in (1, 16))
    block.close()
