"""A given stream: what a call allocates belongs to that stream."""
import pytest
import torch

from tests import _kv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
def test_allocations(monkeypatch, raw):
    from routed_expert_ffn_topk_gb300 import estream as es
    c = _kv.Case([30000, 10], 2, 64, 16, "bf16")
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(2, 4, 64, device="cuda", generator=g).bfloat16()
    k = torch.randn(2, 2, 64, device="cuda", generator=g).bfloat16()
    inv = torch.ones(16, device="cuda")
    logits, u = torch.randn(2, 3000, device="cuda", generator=g), torch.rand(2, device="cuda", generator=g)
    assert c.cache.attend_workspace_bytes(2, 4, c.table.shape[1]) > 0
    side = torch.cuda.Stream()
    at = side.cuda_stream if raw else side
    positions = torch.tensor([100, 5], dtype=torch.int32, device="cuda")
    calls = (lambda **kw: es.kv_append(c.cache, k, k, positions, c.table, q=q, inv_freq=inv, **kw),
             lambda **kw: es.kv_attend(c.cache, q, c.table, c.lens, **kw),
             lambda **kw: es.sample_tokens(logits, u, top_p=0.9, **kw))
    made, empty = [], torch.empty

    def watched(*a, **kw):
        made.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        monkeypatch.setattr(torch, "empty", watched)
        before = len(made)
        got = call(stream=at)
        monkeypatch.setattr(torch, "empty", empty)
        assert len(made) > before and set(made) == {side.cuda_stream}
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
        side.synchronize()
        assert torch.equal(got, want)
    zero = calls[1](stream=0)  # the default stream's handle
    torch.cuda.synchronize()
    assert torch.equal(zero, calls[1]())
