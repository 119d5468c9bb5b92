"""The compiled part of the binding, without a GPU: whatever is not on the call's device goes back to Python."""
import ctypes

import torch

from routed_expert_ffn_topk_gb300 import build as build_mod


def test_gives_back():
    build_mod.build()
    from routed_expert_ffn_topk_gb300 import estream as es
    es.lib()
    f = es._fast
    assert f is not None
    c = es.KvCache(None, None, es.KV_BF16, 0, 16, 2, 64, 1.0, 1.0, 2048, 128, 64, 2048, 128, 64)
    at = ctypes.addressof(c)
    x, n, t = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 1, dtype=torch.int32)
    assert f.kv_append(at, 0, x, x, n, t, None, None, None, False, None) is None
    assert f.kv_append(at, 0, None, 3, "x", t, n, x, n, True, x) is None
    assert f.kv_attend(at, 0, x, t, n, 1.0, 0, x, None, None) is None
    assert f.kv_attend(at, 0, None, t, n, 1.0, 0, x, None, None) is None
    logits, u = torch.zeros(2, 9), torch.zeros(2)
    assert f.sample(0, logits, u, 1.0, 0, 1.0, 0.0, n, None) is None
    assert f.sample(-1, logits, u, 1.0, 0, 1.0, 0.0, n, None) is None
    assert f.sample(0, "logits", None, 1.0, 0, 1.0, 0.0, n, u) is None
    for call in (f.kv_append, f.kv_attend, f.sample):
        assert call() is None and call(at) is None
