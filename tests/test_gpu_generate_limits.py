"""What the token loop refuses and follows: random numbers that are missing or of another shape, and choices that
change; and its attention's end."""
import pytest
import torch

from tests.test_gpu_generate_attention import SAMPLING, _build

pytestmark = pytest.mark.gpu


def test_random_numbers_of_a_run():
    from routed_expert_ffn_topk_gb300 import generate as G
    cfg, experts, loop = _build(sampling=SAMPLING)
    try:
        g = torch.Generator().manual_seed(5)
        prompt = torch.randint(0, 500, (3, 6), generator=g).cuda()
        u = torch.rand(6, 3, generator=g).cuda()
        ids = G.generate(cfg, experts, loop, prompt, 6, u)  # captures
        for bad in (None, u[:1], u[:, :1], u[:, 0], u.double().cpu().tolist()):
            with pytest.raises(ValueError):
                loop.run(ids[:, 0], 5, bad)
        # refused before anything ran: the same run is still to be had
        first = G.generate(cfg, experts, loop, prompt, 1, u[:1])[:, 0]
        assert torch.equal(loop.run(first, 5, u[1:]), ids[:, 1:])
    finally:
        loop.stack.close()


def test_other_choices_than_captured():
    """A loop whose choices change after a run takes the new ones."""
    from routed_expert_ffn_topk_gb300 import generate as G
    cfg, experts, loop = _build()
    try:
        g = torch.Generator().manual_seed(6)
        prompt, u = torch.randint(0, 500, (3, 6), generator=g).cuda(), torch.rand(7, 3, generator=g).cuda()
        likeliest = G.generate(cfg, experts, loop, prompt, 7)
        loop.sampling = dict(temperature=1.5)
        drawn = G.generate(cfg, experts, loop, prompt, 7, u)
        G.generate(cfg, experts, loop, prompt, 1, u[:1])
        now = drawn[:, 0]
        for i in range(1, 7):
            now = loop.step(now, u[i])
            assert torch.equal(now, drawn[:, i]), i
        loop.sampling["temperature"] = 0.0
        assert torch.equal(G.generate(cfg, experts, loop, prompt, 7, u), likeliest)
        loop.sampling = None
        assert torch.equal(G.generate(cfg, experts, loop, prompt, 7), likeliest)
        assert torch.equal(G.generate(cfg, experts, loop, prompt, 7, u), likeliest)  # no use for u
    finally:
        loop.stack.close()


def test_tokens_past_the_end():
    from routed_expert_ffn_topk_gb300 import generate as G
    cfg, experts, loop = _build(tokens=20)
    try:
        a = loop.attention
        prompt = torch.randint(0, 500, (3, 10), generator=torch.Generator().manual_seed(7)).cuda()
        ids = G.generate(cfg, experts, loop, prompt, 6)  # holds 15
        with pytest.raises(ValueError):
            loop.run(ids[:, -1], 6)
        assert a.lens.tolist() == [15] * 3
        more = loop.run(ids[:, -1], 5)
        assert int(more.min()) >= 0 and a.lens.tolist() == [20] * 3
        X = torch.zeros(3, cfg.H, dtype=torch.bfloat16, device="cuda")
        for call in (lambda: loop.run(more[:, -1], 1), lambda: loop.step(more[:, -1]), lambda: a.step(X)):
            with pytest.raises(ValueError):
                call()
        assert a.lens.tolist() == [20] * 3
        # a caller that sets the lengths back has the room again, by whichever reference
        lens = a.lens
        lens.fill_(19)
        a.step(X)
        with pytest.raises(ValueError):
            a.step(X)
        lens.fill_(18)
        a.step(X)
        # one long sequence is enough for a refusal
        a.lens.copy_(torch.tensor([3, 20, 4], dtype=torch.int32))
        with pytest.raises(ValueError):
            a.step(X)
        assert torch.equal(G.generate(cfg, experts, loop, prompt, 6), ids)
    finally:
        loop.stack.close()
