"""Attention's precision where the formula needs every bit of a weight."""
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
