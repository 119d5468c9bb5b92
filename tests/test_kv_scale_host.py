"""Attention's scale: refused where its factor to base 2 leaves fp32 (every score would be infinite or NaN)."""
import ctypes

import pytest

from routed_expert_ffn_topk_gb300 import build as build_mod


@pytest.mark.parametrize("scale,k_scale,ok", [(2.3e38, 1.0, True), (-2.3e38, 1.0, True), (2.4e38, 1.0, False), (-3e38, 1.0, False),
                                              (1e8, 2.0 ** 100, True), (1e9, 2.0 ** 100, False), (1e30, 2.0 ** -100, True)])
def test_range(scale, k_scale, ok):
    build_mod.build()
    from routed_expert_ffn_topk_gb300 import estream as es
    p = 1 << 20  # never read: no rows
    c = es.KvCache(p, p, es.KV_E4M3, 4, 16, 2, 64, k_scale, 1.0, 2048, 128, 64, 2048, 128, 64)
    st = es.lib().estream_kv_attend(ctypes.byref(c), es.KV_BF16, 0, 4, None, 256, 64, None, 1, 1, None, scale, 0, None, 256, 64, None,
                                    None, 0, None)
    assert st == (es.OK if ok else es.ERR_INVALID_ARG)
