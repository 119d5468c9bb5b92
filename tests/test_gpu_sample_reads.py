"""Sampling without cuts at sizes where a lane reads many parts of a row: what is read again is found from each
part's largest logit. Tokens as in exact arithmetic; probabilities within 2^-23 (see test_gpu_sample)."""
import pytest
import torch

from tests.test_gpu_sample import _es, check, want

pytestmark = pytest.mark.gpu

KINDS = 8


def _rows(V, dtype, seed):
    """Rows of different density: flat, peaked, one finite logit at either end, runs of equal ones, mostly masked."""
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(KINDS, V, generator=g) * 2.0
    l[1, torch.randint(0, V, (5,), generator=g)] += 12.0
    l[2], l[3] = float("-inf"), float("-inf")
    l[2, 0], l[3, V - 1] = 1.5, -3.0
    l[4, V // 3:] = 1.0
    l[5, torch.rand(V, generator=g) < 0.99] = float("-inf")
    l[6] = torch.linspace(-30, 5, V)
    l[7] = 0.25
    return l.to(dtype), torch.rand(KINDS, 4, generator=g)


@pytest.mark.parametrize("V,dtype,ld", [(100003, torch.float32, 100008), (100003, torch.float32, 100003),
                                        (393216, torch.bfloat16, 393216), (65541, torch.float16, 65544), (2051, torch.float32, 2052)])
@pytest.mark.parametrize("kw", [dict(min_p=0.3), dict(min_p=0.02, temperature=1.4), dict(min_p=1e-7), dict(temperature=0.0), dict()])
def test_many_rows(V, dtype, ld, kw):
    """640 rows, a CTA each: KINDS rows 80 times over."""
    es, times = _es(), 80
    l, u = _rows(V, dtype, V % 97)
    big = torch.zeros(KINDS * times, ld, dtype=dtype, device="cuda")
    big[:, :V] = l.cuda().repeat(times, 1)
    us = u.t().reshape(-1).repeat(times // 4)  # row r of copy c: u[r, c % 4]
    prob = torch.empty(KINDS * times, device="cuda")
    ids = es.sample_tokens(big[:, :V], us.cuda(), prob=prob, **kw)
    wi, wp = want(l.repeat(4, 1), us[:4 * KINDS], **kw)
    assert torch.equal(ids.cpu(), wi.repeat(times // 4))
    p = prob.cpu().double().view(times // 4, -1)
    assert bool(((p - wp).abs() <= wp * 2.0 ** -23).all())


@pytest.mark.parametrize("B", [1, 70, 160])
@pytest.mark.parametrize("kw", [dict(min_p=0.1), dict(temperature=0.0), dict()])
def test_clusters(B, kw):
    """Fewer rows, split over clusters of 8 and fewer CTAs."""
    l, u = _rows(30011, torch.float32, B)
    times = -(-B // KINDS)
    check(l.repeat(times, 1)[:B].cuda(), u.t().reshape(-1).repeat(-(-times // 4))[:B].cuda(), **kw)
