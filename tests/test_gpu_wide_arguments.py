"""Numbers past 32 bits are refused, not cut to their low bits."""
import pytest
import torch

from tests import _kv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 5])
def test_wide_numbers(n):
    from routed_expert_ffn_topk_gb300 import estream as es
    c = _kv.Case([30, 10], 2, 64, 16, "bf16")
    q = torch.zeros(2, 4, 64, device="cuda").bfloat16()
    es.kv_attend(c.cache, q, c.table, c.lens, window=(1 << 31) - 1)
    with pytest.raises(ValueError):
        es.kv_attend(c.cache, q, c.table, c.lens, window=n)
    logits, u = torch.randn(2, 100, device="cuda"), torch.rand(2, device="cuda")
    es.sample_tokens(logits, u, top_k=(1 << 31) - 1)
    with pytest.raises(ValueError):
        es.sample_tokens(logits, u, top_k=n)
