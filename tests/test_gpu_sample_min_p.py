"""min-p above 1: only the largest logit is kept, and of equal ones the first, as where top-p is 0."""
import pytest
import torch

from tests import test_gpu_sample as S

pytestmark = pytest.mark.gpu


def _tied(B, V, dtype, n):
    """Rows whose n largest logits are equal, at places spread over the row."""
    l, u = S.rows(B, V, seed=V + n, dtype=dtype)
    g = torch.Generator().manual_seed(n)
    for b in range(B):
        l[b, torch.randperm(V, generator=g)[:n].cuda()] = 20.0
    return l, u


@pytest.mark.parametrize("min_p", [1.0, 1.0 + 2.0 ** -23, 2.0, float("inf")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,n", [(50, 2), (3000, 7), (40000, 200), (40000, 5000)])
def test_tied_largest(min_p, dtype, V, n):
    l, u = _tied(9, V, dtype, n)
    for kw in (dict(), dict(top_k=5), dict(top_k=1500), dict(top_p=0.6), dict(top_p=0.9, top_k=V - 1), dict(temperature=0.3)):
        ids = S.check(l, u, min_p=min_p, **kw)
        if min_p > 1:
            assert torch.equal(ids.long(), (l == l.amax(1, keepdim=True)).int().argmax(1))


def test_a_choice_a_row():
    l, u = _tied(12, 9000, torch.bfloat16, 30)
    m = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, float("inf")] * 2, device="cuda")
    S.check(l, u, min_p=m)
    S.check(l, u, min_p=m, top_k=torch.tensor([0, 4, 0, 4, 0, 4] * 2, dtype=torch.int32, device="cuda"))
    S.check(l, u, min_p=m, top_p=torch.tensor([0.5, 1.0] * 6, device="cuda"))
