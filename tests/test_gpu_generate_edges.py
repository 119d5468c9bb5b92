"""The 4-bit prompt layer at the ends of its sizes."""
import pytest
import torch

from tests.test_gpu_generate import _layer

pytestmark = pytest.mark.gpu


def test_no_tokens():
    from routed_expert_ffn_topk_gb300 import generate as G
    layer = G.Mx4Experts(*_layer())
    X = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    Y = layer.prefill(X, torch.empty(0, 8, device="cuda"), 2, False)
    assert Y.shape == (0, 256) and Y.dtype == torch.float32
