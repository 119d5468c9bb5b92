"""The legacy default stream by its handles, 0 and 1 (cudaStreamLegacy): calls allocate and run there."""
import pytest
import torch

from tests import _kv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [0, 1])
def test_handle(monkeypatch, handle):
    from routed_expert_ffn_topk_gb300 import estream as es
    c = _kv.Case([30000, 10], 2, 64, 16, "bf16")
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(2, 4, 64, device="cuda", generator=g).bfloat16()
    logits, u = torch.randn(2, 3000, device="cuda", generator=g), torch.rand(2, device="cuda", generator=g)
    x = torch.randn(70, 256, device="cuda", generator=g).bfloat16()
    calls = (lambda **kw: es.kv_attend(c.cache, q, c.table, c.lens, **kw),
             lambda **kw: es.sample_tokens(logits, u, top_p=0.9, **kw),
             lambda **kw: es.mx4_dequantize(es.mx4_quantize(x, es.FP4_E4M3X16, 0.01, **kw), **kw))
    want = [call() for call in calls]
    made, empty = [], torch.empty

    def watched(*a, **kw):
        made.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        monkeypatch.setattr(torch, "empty", watched)
        got = [call(stream=handle) for call in calls]
        monkeypatch.setattr(torch, "empty", empty)
    torch.cuda.synchronize()
    assert made and set(made) == {0}
    assert all(torch.equal(a, b) for a, b in zip(got, want))
