"""The path that runs the few-token layer and the 4-bit calls together.

Tolerances: the 4-bit layer against the same steps with fp64 products. The sums
differ by about 1e-6, which moves a bf16 gate or up value, and through it a code of
h by one step (at most half its value), in about 1e-3 of the values; in the 2-norm
that is sqrt(1e-3) / 2 = 1.6e-2 of h at the very most, and REL = 2e-2 of Y."""
import pytest
import torch

pytestmark = pytest.mark.gpu

REL = 2e-2


def _layer(E=8, F=192, H=256, seed=3):
    g = torch.Generator().manual_seed(seed)
    f = lambda *s: (torch.randn(*s, generator=g) / s[-1] ** 0.5).to(torch.bfloat16)
    return f(E, F, H), f(E, F, H), f(E, H, F)


def _wide(w, es, fmt):
    """The fp64 values of a weight's quantised rows."""
    rows = w.reshape(-1, w.shape[-1]).cuda()
    q = es.mx4_quantize(rows, fmt, es.mx4_tensor_scale(float(rows.abs().max()), fmt))
    return es.mx4_dequantize(q).double().view(w.shape)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("T,k,renorm", [(1, 2, False), (37, 2, True), (900, 3, False)])
def test_prompt_layer(fmt, T, k, renorm):
    from routed_expert_ffn_topk_gb300 import estream as es
    from routed_expert_ffn_topk_gb300 import generate as G
    Wg, Wu, Wd = _layer()
    layer = G.Mx4Experts(Wg, Wu, Wd, fmt)
    g = torch.Generator().manual_seed(T)
    X = torch.randn(T, 256, generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn(T, 8, generator=g).cuda()
    logits[:, 5] = -1e30  # an expert without tokens
    Y = layer.prefill(X, logits, k, renorm)
    assert torch.equal(Y, layer.prefill(X, logits, k, renorm))
    gu, down = _wide(torch.cat([Wg, Wu], 1), es, fmt), _wide(Wd, es, fmt)
    xd = es.mx4_dequantize(es.mx4_quantize(X, fmt, layer.act_scale)).double()
    p = torch.softmax(logits.double(), -1)
    a, ids = p.topk(k, -1)
    if renorm:
        a = a / a.sum(-1, keepdim=True)
    want = torch.zeros(T, 256, dtype=torch.float64, device="cuda")
    for j in range(k):
        for e in range(8):
            t = (ids[:, j] == e).nonzero()[:, 0]
            if t.numel():
                v = (xd[t] @ gu[e].t()).to(torch.bfloat16)
                h = es.mx4_dequantize(es.mx4_quantize(v, fmt, layer.act_scale, swiglu=True)).double()
                want[t] += a[t, j, None] * (h @ down[e].t())
    assert float((Y.double() - want).norm() / want.norm()) <= REL
    with pytest.raises(ValueError):
        layer.prefill(X[:, :128], logits, k, renorm)


def test_prompt_and_tokens():
    """The replayed steps give the tokens of the same calls made one by one."""
    from routed_expert_ffn_topk_gb300 import estream as es
    from routed_expert_ffn_topk_gb300 import generate as G
    from routed_expert_ffn_topk_gb300 import workloads as W
    import dataclasses
    saved = dict(W.CONFIGS)
    W.CONFIGS["small"] = dataclasses.replace(W.CONFIGS["c2"], H=256, E=8, k=2, F=128, G=8, B=1, P=8)
    try:
        cfg, experts, loop = G.build("small", 3, 500)
    finally:
        W.CONFIGS.clear()
        W.CONFIGS.update(saved)
    try:
        prompt = torch.randint(0, 500, (3, 20), generator=torch.Generator().manual_seed(1)).cuda()
        ids = G.generate(cfg, experts, loop, prompt, 6)
        assert tuple(ids.shape) == (3, 6) and int(ids.min()) >= 0 and int(ids.max()) < 500
        now = ids[:, 0]
        for i in range(1, 6):
            now = loop.step(now)
            assert torch.equal(now, ids[:, i]), i
        assert torch.equal(G.generate(cfg, experts, loop, prompt, 6), ids)
        assert es.get_device_error(loop.stack.ctx) == es.OK and es.mx4_error() == es.OK
    finally:
        loop.stack.close()
