"""A given stream: what the 4-bit, router and route calls allocate, to work in or to return, belongs to that stream."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _flat(x):
    if isinstance(x, torch.Tensor):
        return [x]
    if isinstance(x, dict):
        return [x[k] for k in sorted(x) if k != "workspace"]
    return [x.codes, x.scales] if hasattr(x, "scales") else [x.tiles]


@pytest.mark.parametrize("raw", [False, True])
def test_allocations(monkeypatch, raw):
    from routed_expert_ffn_topk_gb300 import estream as es
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(70, 256, device="cuda", generator=g).bfloat16()
    W_r = torch.randn(8, 256, device="cuda", generator=g).bfloat16()
    logits = torch.randn(70, 8, device="cuda", generator=g)
    x4 = es.mx4_quantize(x, es.FP4_E4M3X16, 0.01)
    w4 = es.mx4_weights(x4.codes, x4.scales, 256, es.FP4_E4M3X16, 0.01)
    calls = (lambda **kw: es.mx4_quantize(x, es.FP4_E4M3X16, 0.01, **kw),
             lambda **kw: es.mx4_dequantize(x4, **kw),
             lambda **kw: es.mx4_weights(x4.codes, x4.scales, 256, es.FP4_E4M3X16, 0.01, **kw),
             lambda **kw: es.mx4_product(x4, w4, **kw),
             lambda **kw: es.route_build(logits, 2, True, **kw),
             lambda **kw: es.router_logits(x, W_r, **kw),
             lambda **kw: es.route_build_from_x(x, W_r, 2, True, **kw),
             lambda **kw: es.route_build_noalloc(logits, 2, True, **kw))
    side = torch.cuda.Stream()
    at = side.cuda_stream if raw else side
    made, empty = [], torch.empty

    def watched(*a, **kw):
        made.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)
    for i, call in enumerate(calls):
        want = _flat(call())
        torch.cuda.synchronize()
        monkeypatch.setattr(torch, "empty", watched)
        before = len(made)
        got = call(stream=at)
        monkeypatch.setattr(torch, "empty", empty)
        assert len(made) > before and set(made) == {side.cuda_stream}, i
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(_flat(got), want)), i


def test_layer_from_router(monkeypatch):
    """The buffer that a layer stack keeps for its router's logits."""
    from tests.test_gpu_generate_attention import _build
    cfg, experts, loop = _build()
    try:
        g = torch.Generator(device="cuda").manual_seed(2)
        X = torch.randn(3, cfg.H, device="cuda", generator=g).bfloat16()
        Y, Z = (torch.zeros(3, cfg.H, device="cuda") for _ in range(2))
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        made, empty = [], torch.empty

        def watched(*a, **kw):
            made.append(torch.cuda.current_stream().cuda_stream)
            return empty(*a, **kw)
        monkeypatch.setattr(torch, "empty", watched)
        logits = loop.stack.prefill_from_router(0, X, loop.W_r, Y, stream=side)
        monkeypatch.setattr(torch, "empty", empty)
        assert made and set(made) == {side.cuda_stream}
        side.synchronize()
        kept = logits.clone()
        again = loop.stack.prefill_from_router(0, X, loop.W_r, Z)
        torch.cuda.synchronize()
        assert torch.equal(again, kept) and torch.equal(Y, Z)
    finally:
        loop.stack.close()
