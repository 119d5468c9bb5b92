"""Attention over infinite values."""
import math

import pytest
import torch

from tests import _kv
from tests.test_gpu_kv_attend import _q

pytestmark = pytest.mark.gpu


def _es():
    from routed_expert_ffn_topk_gb300 import estream as es
    return es


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("lens", [[60, 33], [30000, 50]])
def test_infinite_values(kind, lens):
    """An attended infinite value makes its column of the heads that meet it infinite or NaN, and nothing
    else. Both forms: a cluster a unit, and shares that are joined."""
    es = _es()
    c = _kv.Case(lens, 2, 64, 16, kind)
    q = _q(2, 6, 64, kind)
    M = c.table.shape[1]
    assert (c.cache.attend_workspace_bytes(2, 6, M) > 0) == (max(lens) > 1000)
    good = es.kv_attend(c.cache, q, c.table, c.lens)
    p, s = c.place[0]
    for at, d, sign in ((0, 5, 1), (len(p) // 2, 17, -1), (len(p) - 1, 63, 1)):
        c.v[p[at], s[at], 1, d] = sign * math.inf
    lse = torch.zeros(2, 6, device="cuda")
    out = es.kv_attend(c.cache, q, c.table, c.lens, lse=lse)
    hit = torch.zeros(2, 6, 64, dtype=torch.bool, device="cuda")
    hit[0, 3:, [5, 17, 63]] = True
    assert not bool(out[hit].isfinite().any()) and bool(lse.isfinite().all())
    assert torch.equal(out[~hit], good[~hit])


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("n", [60, 30000])
def test_infinite_score(kind, n):
    """A score of +infinity makes its heads' rows and lse NaN, and leaves the others."""
    es = _es()
    c = _kv.Case([n, 40], 2, 64, 16, kind)
    q = _q(2, 6, 64, kind).abs()
    want = es.kv_attend(c.cache, q, c.table, c.lens)
    p, s = c.place[0]
    c.k[p[n // 3], s[n // 3], 0, 9] = math.inf
    lse = torch.zeros(2, 6, device="cuda")
    out = es.kv_attend(c.cache, q, c.table, c.lens, lse=lse)
    assert bool(out[0, :3].isnan().all()) and bool(lse[0, :3].isnan().all())
    assert torch.equal(out[0, 3:], want[0, 3:]) and torch.equal(out[1], want[1])
    assert bool(lse[0, 3:].isfinite().all()) and bool(lse[1].isfinite().all())
