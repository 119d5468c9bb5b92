"""The path that runs the paged cache, attention and sampling with the layer's calls."""
import dataclasses

import pytest
import torch

pytestmark = pytest.mark.gpu


def _build(batch=3, vocab=500, tokens=40, sampling=None):
    from routed_expert_ffn_topk_gb300 import generate as G
    from routed_expert_ffn_topk_gb300 import workloads as W
    saved = dict(W.CONFIGS)
    W.CONFIGS["small"] = dataclasses.replace(W.CONFIGS["c2"], H=512, E=8, k=2, F=128, G=8, B=1, P=8)
    try:
        return G.build("small", batch, vocab, attend_tokens=tokens, sampling=sampling)
    finally:
        W.CONFIGS.clear()
        W.CONFIGS.update(saved)


SAMPLING = dict(temperature=0.9, top_k=40, top_p=0.9, min_p=0.01)


@pytest.mark.parametrize("sampling", [None, SAMPLING])
def test_prompt_and_tokens(sampling):
    """The replayed steps give the tokens of the same calls made one by one, and the same again."""
    from routed_expert_ffn_topk_gb300 import estream as es
    from routed_expert_ffn_topk_gb300 import generate as G
    cfg, experts, loop = _build(sampling=sampling)
    try:
        g = torch.Generator().manual_seed(1)
        prompt = torch.randint(0, 500, (3, 20), generator=g).cuda()
        u = torch.rand(8, 3, generator=g).cuda() if sampling else None
        ids = G.generate(cfg, experts, loop, prompt, 8, u)
        assert tuple(ids.shape) == (3, 8) and int(ids.min()) >= 0 and int(ids.max()) < 500
        assert loop.attention.lens.tolist() == [27] * 3
        assert torch.equal(G.generate(cfg, experts, loop, prompt, 8, u), ids)
        G.generate(cfg, experts, loop, prompt, 1, None if u is None else u[:1])  # the prompt's keys again
        now = ids[:, 0]
        for i in range(1, 8):
            now = loop.step(now, None if u is None else u[i])
            assert torch.equal(now, ids[:, i]), i
        assert es.get_device_error(loop.stack.ctx) == es.OK and es.mx4_error() == es.OK
        with pytest.raises(ValueError):
            G.generate(cfg, experts, loop, prompt, 22, None if u is None else u.new_zeros(22, 3))
        if sampling:
            with pytest.raises(ValueError):
                G.generate(cfg, experts, loop, prompt, 8)
    finally:
        loop.stack.close()


def test_greedy_is_temperature_0():
    from routed_expert_ffn_topk_gb300 import generate as G
    cfg, experts, loop = _build()
    try:
        prompt = torch.randint(0, 500, (3, 9), generator=torch.Generator().manual_seed(2)).cuda()
        ids = G.generate(cfg, experts, loop, prompt, 5)
        loop.sampling, loop.graph = dict(temperature=0.0), None
        assert torch.equal(G.generate(cfg, experts, loop, prompt, 5, torch.rand(5, 3, device="cuda")), ids)
    finally:
        loop.stack.close()


def test_prompt_in_one_call_or_token_by_token():
    """Attention's rows of a prompt are those of its tokens one at a time. The two calls split a row's positions
    differently: sums differ by 2^-12 of the mean magnitude at most (tests/_kv.py), which moves a bf16 result by a
    step (2^-7) at most; a 4-bit code of the projection's input then moves by one, at most half its value, in
    one value of 30 (2^-7 of the spacing 1/4): sqrt(1 / 30) / 2 = 0.09 of the 2-norm at the very most."""
    cfg, experts, loop = _build(batch=2, tokens=70)
    try:
        a = loop.attention
        X = torch.randn(2 * 65, cfg.H, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
        whole = a.prefill(X, 65).view(2, 65, -1).float()
        k, v = a.cache.k.clone(), a.cache.v.clone()
        a.lens.zero_()
        rows = X.view(2, 65, -1)
        steps = torch.stack([a.step(rows[:, i].contiguous()) for i in range(65)], 1).float()
        assert torch.equal(a.cache.k, k) and torch.equal(a.cache.v, v)
        assert float((steps - whole).norm() / whole.norm()) <= 0.09
        with pytest.raises(ValueError):
            a.prefill(X, 64)
    finally:
        loop.stack.close()
