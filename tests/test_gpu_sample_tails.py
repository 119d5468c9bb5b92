"""Rows with many tokens far below the largest: the header's bound on where u may lie beside the token's own share.

A weight is held to 2^-37 of itself and rounded to a unit of 2^-45 of the largest, by half a unit at most, so the sum up to
any token is off by 2^-37 of the kept weight and by V 2^-46 of the largest; and so is the whole, which u multiplies, with the
other sign at worst: the difference of the two has each token's error once, times u or 1 - u. One unit more for the
product's rounding, and V 2^-52 for this test's own sums in 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _check(l, u, temperature=1.0, top_k=0):
    """The drawn token's exact share of [0, 1), widened by the bound, holds u."""
    from routed_expert_ffn_topk_gb300 import estream as es
    ids = es.sample_tokens(l, u, temperature=temperature, top_k=top_k).cpu().long()
    V = l.shape[1]
    bound = 2.0 ** -37 + V * 2.0 ** -46 + 2.0 ** -45 + V * 2.0 ** -52
    for b, i in enumerate(ids.tolist()):
        x = l[b].double().cpu()
        w = torch.exp((x - x.max()) / float(torch.tensor(temperature)))
        if top_k:
            w[torch.argsort(x, descending=True, stable=True)[top_k:]] = 0.0
        upto = w.cumsum(0) / w.sum()
        before = float(upto[i - 1]) if i else 0.0
        assert w[i] > 0 and before - bound <= float(u[b]) <= float(upto[i]) + bound, (b, i, before, float(u[b]), float(upto[i]))


@pytest.mark.parametrize("top_k", [0, 300000])
@pytest.mark.parametrize("last", [False, True])
def test_half_units(last, top_k):
    """Weights that lie between two units add up their roundings: 393215 of 2^-41.42 behind, or before, the largest."""
    V = 393216
    l = torch.full((1, V), -28.713, device="cuda")
    l[0, V - 1 if last else 0] = 0.0
    us = [1.5e-8, 1.0e-7, 1.2e-7, 1.25e-7, 1.3e-7] if last else [1 - 2.0 ** -24, 1 - 2.0 ** -23, 1 - 1.5 * 2.0 ** -23, 1 - 2.0 ** -22]
    _check(l.expand(len(us), V), torch.tensor(us, device="cuda"), top_k=top_k)


@pytest.mark.parametrize("V", [32000, 151936, 393216])
@pytest.mark.parametrize("far", [-27.0, -28.0, -29.11, -30.3])
def test_far_tails(V, far):
    """Tails at other distances, u on both sides of the border between the largest and them."""
    l = torch.full((1, V), far, device="cuda")
    l[0, V // 2] = 0.0
    tail = float(torch.exp(torch.tensor(far, dtype=torch.float64))) * V
    half = tail / 2 / (1 + tail)
    _check(l.expand(4, V), torch.tensor([half * 0.8, half * 1.2, 1 - half * 1.2, 1 - half * 0.8], dtype=torch.float64).float().cuda())
