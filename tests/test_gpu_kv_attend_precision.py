"""Attention's precision where the formula needs every bit of a weight or of the logarithm."""
import math

import pytest
import torch

from tests import _kv

pytestmark = pytest.mark.gpu


def _es():
    from routed_expert_ffn_topk_gb300 import estream as es
    return es

@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("far", [0, 30000])
def test_weights_of_two_terms(kind, far):
    """Two positions of nearly equal score and opposite values: out = tanh(delta / 2), all of which comes from what one weight
    lacks of the other. Scores are exact (one product each), so a weight is off by 2^-22 (exponential, and the rounding of its
    base 2 argument below 2^-7 to 2^-31) and its terms' rounding, 2^-16 for bf16's two and 2^-22 for fp16's: half of their sum
    in out, which is rounded by half a step itself (fp16's smallest step is 2^-24). far: in a long row whose other positions are
    out of sight (e^-60)."""
    es = _es()
    B, dim, n = 40, 16, far + 2
    c = _kv.Case([n] * (B if not far else 3), 1, dim, 16, kind, seed=1)
    B = len(c.lens_list)
    delta = (torch.arange(1, B + 1) * (0.0002 if not far else 0.0012)).to(_kv.DT[kind])
    q = torch.zeros(B, 1, dim, dtype=_kv.DT[kind], device="cuda")
    q[:, 0, 0] = 1.0
    for b in range(B):
        p, s = c.place[b]
        c.k[p, s], c.v[p, s] = 0.0, 1.0
        c.k[p, s, 0, 0] = -60.0
        c.k[p[0], s[0], 0, 0], c.k[p[-1], s[-1], 0, 0] = 0.0, -float(delta[b])
        c.v[p[-1], s[-1]] = -1.0
    out = es.kv_attend(c.cache, q, c.table, c.lens, scale=1.0)[:, 0, 0].double().cpu()
    d = delta.double()
    rest = far * math.exp(-60.0)
    want = (1.0 - torch.exp(-d) + rest) / (1.0 + torch.exp(-d) + rest)
    tol = (2.0 ** -22 + 2.0 ** -31 + (2.0 ** -16 if kind == "bf16" else 2.0 ** -22)) / 2 + want * torch.finfo(q.dtype).eps / 2 + 2.0 ** -25
    assert bool(((out - want).abs() <= tol).all()), (out - want).abs().max()


def test_weights_next_to_8_bits():
    """The same over E4M3 pages: keys of 4 bits and a small scale make the deltas; weights of two fp16 terms."""
    es = _es()
    c = _kv.Case([2] * 64, 1, 16, 16, "e4m3", seed=1)
    size = torch.tensor([(8 + i % 8) * 2.0 ** (i // 8) / 8 for i in range(64)])
    for (p, s), x in zip(c.place, size.tolist()):
        _kv.put(c.k, p, s, torch.tensor([0.0, -x], device="cuda")[:, None, None].expand(2, 1, 16) * (torch.arange(16, device="cuda") == 0))
        _kv.put(c.v, p, s, torch.tensor([1.0, -1.0], device="cuda")[:, None, None].expand(2, 1, 16))
    q = torch.zeros(64, 1, 16, dtype=torch.float16, device="cuda")
    q[:, 0, 0] = 1.0
    out = es.kv_attend(c.cache, q, c.table, c.lens, scale=2.0 ** -13)[:, 0].double().cpu()
    want = torch.tanh(size.double() * 2.0 ** -14)[:, None]
    tol = (2.0 ** -22 + 2.0 ** -31 + 2.0 ** -22) / 2 + want * 2.0 ** -11 + 2.0 ** -25
    assert bool(((out - want).abs() <= tol).all()), (out - want).abs().max()


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
def test_log_sum_of_one_position(kind):
    """lse of one position is its score. The product is exact; it is rounded once where it meets the factor to base 2 and once
    where it comes back, each by half a step, 2^-24 of the score: 2^-23, and 2^-30 for what the factors' second terms leave.
    The score's part behind the whole number goes through an exponential, within 2^-22, and a logarithm to base 2 of a value
    between 1/2 and 1, within 2^-24: (1.45 2^-22 + 2^-24) ln 2 and the product's rounding, together below 2^-21."""
    es = _es()
    c = _kv.Case([1] * 64, 1, 16, 16, kind, scales=(0.75, 1.0) if kind == "e4m3" else (1.0, 1.0))
    # values of up to 7 bits, of 4 for E4M3
    size = torch.tensor([(8 + i % 8) * 2.0 ** (i // 8) / 8 if kind == "e4m3" else 33.0 + i for i in range(64)])
    for (p, s), x in zip(c.place, size.tolist()):
        _kv.put(c.k, p, s, torch.full((1, 1, 16), x, device="cuda"))
    q = torch.ones(64, 1, 16, dtype=torch.bfloat16 if kind == "e4m3" else _kv.DT[kind], device="cuda")
    for i in range(24):
        scale = (-1) ** i * 0.37 * 1.173 ** i
        lse = torch.zeros(64, 1, device="cuda")
        es.kv_attend(c.cache, q, c.table, c.lens, scale=scale, lse=lse)
        want = 16.0 * size.double() * float(torch.tensor(scale)) * c.scales[0]
        far = (lse[:, 0].double().cpu() - want).abs()
        assert bool((far <= want.abs() * (2.0 ** -23 + 2.0 ** -30) + 2.0 ** -21).all()), (scale, float((far / want.abs()).max()) * 2.0 ** 24)


def test_log_sum_without_a_scale():
    """scale 0: every score is 0, and lse the logarithm of how many there are, a logarithm to base 2 (within one step, 2^-23)
    times ln 2 (rounded, as the product is: 2^-24 each)."""
    es = _es()
    c = _kv.Case([1, 7, 1000, 30000], 2, 64, 16, "f16")
    lse = torch.zeros(4, 4, device="cuda")
    es.kv_attend(c.cache, torch.ones(4, 4, 64, dtype=torch.float16, device="cuda"), c.table, c.lens, scale=0.0, lse=lse)
    want = c.lens.double().cpu().log()[:, None]
    assert bool(((lse.double().cpu() - want).abs() <= want * 2.0 ** -22 + 2.0 ** -30).all())
