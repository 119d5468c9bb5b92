"""What the rotation leaves as it is: values behind the rotated part, whatever stands beside them; and pairs
whose frequency is no number."""
import pytest
import torch

from tests import _kv

pytestmark = pytest.mark.gpu


def _append(x, dim, rot, kind, interleaved, inv_freq=None):
    """Rows x [T, 2, dim] as keys, values and queries at positions 3, 4, ...: the cache's keys and values, and the queries."""
    from routed_expert_ffn_topk_gb300 import estream as es
    T = x.shape[0]
    k, v = _kv.pages(2, 16, 2, dim, kind, fill=3.0), _kv.pages(2, 16, 2, dim, kind, fill=3.0)
    positions = torch.arange(3, 3 + T, dtype=torch.int32, device="cuda")
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda").expand(T, 1)
    f = torch.full((rot // 2,), 0.3, device="cuda") if inv_freq is None else inv_freq
    q = es.kv_append(es.PagedKV(k, v), x, x, positions, table, q=x, inv_freq=f, interleaved=interleaved)
    return k[1, 3:3 + T], v[1, 3:3 + T], q


def _same(a, b):
    """Equal, zeros by their sign too, NaN as NaN."""
    a, b = a.float(), b.float()
    return bool(((a == b) & (a.signbit() == b.signbit()) | a.isnan() & b.isnan()).all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("dim,rot", [(32, 2), (64, 6), (64, 12), (128, 20), (128, 126), (128, 64), (64, 0)])
@pytest.mark.parametrize("off", [0, 1])
def test_unrotated_values(interleaved, kind, dim, rot, off):
    """Infinities, NaN and zeros of either sign behind the rotated part, each next to each of them; off 1: rows off 16 bytes."""
    inf = float("inf")
    x = torch.randn(6, 2, dim, generator=torch.Generator().manual_seed(rot)).bfloat16() if kind != "f16" else \
        torch.randn(6, 2, dim, generator=torch.Generator().manual_seed(rot)).half()
    some = torch.tensor([1.5, -1.0, inf, -0.0, -inf, 0.25, float("nan"), -2.0])
    n = dim - rot
    for t in range(6):
        x[t, :, rot:] = some[(torch.arange(n) * (1 + t) + t) % 8].to(x.dtype)
    wide = torch.zeros(6, 2, dim + off, dtype=x.dtype)
    wide[..., off:] = x
    x = wide.cuda()[..., off:]
    k, v, q = _append(x, dim, rot, kind, interleaved)
    want = x[..., rot:]
    assert _same(q[..., rot:], want)
    if kind == "e4m3":
        want = want.float().clamp(-448.0, 448.0)
    assert _same(k[..., rot:], want) and _same(v[..., rot:], want)
    assert bool(q[..., :rot].isfinite().all()) and bool(k[..., :rot].float().isfinite().all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 20), (128, 64)])
def test_frequencies_that_are_no_numbers(interleaved, dim, rot):
    """An infinite or NaN frequency makes its pair NaN, as sine and cosine of it are, and leaves the others."""
    x = torch.randn(4, 2, dim, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    f = torch.full((rot // 2,), 0.3, device="cuda")
    k0, _, q0 = (t.clone() for t in _append(x, dim, rot, "bf16", interleaved, f))
    for j, bad in ((0, float("inf")), (rot // 2 - 1, float("nan")), (3, -float("inf"))):
        f[j] = bad
    k, _, q = _append(x, dim, rot, "bf16", interleaved, f)
    hit = torch.zeros(dim, dtype=torch.bool, device="cuda")
    for j in (0, 3, rot // 2 - 1):
        hit[[2 * j, 2 * j + 1] if interleaved else [j, j + rot // 2]] = True
    for got, plain in ((k, k0), (q, q0)):
        assert bool(got[..., hit].isnan().all()) and torch.equal(got[..., ~hit], plain[..., ~hit])
