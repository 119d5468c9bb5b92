"""Sampling from given random numbers against its definition in 64 bits. Tokens have to be equal; a probability is a
quotient of sums that hold 2^-38 of each weight, rounded to fp32: 2^-24 of itself, and 2^-23 is asked."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _es():
    from routed_expert_ffn_topk_gb300 import estream as es
    return es


def want(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """ids, prob of rows on the CPU, in 64 bits."""
    B, V = logits.shape
    f32 = lambda x, b: float(x[b]) if torch.is_tensor(x) else float(torch.tensor(x, dtype=torch.float32))
    ids, probs = [], []
    for b in range(B):
        l = logits[b].double().cpu()
        t, p, low, r = f32(temperature, b), f32(top_p, b), f32(min_p, b), f32(u, b)
        k = int(top_k[b]) if torch.is_tensor(top_k) else top_k
        if bool(l.isnan().any()) or not math.isfinite(float(l.max())):
            ids.append(-1)
            probs.append(math.nan)
            continue
        if not t > 2.0 ** -100:
            ids.append(int((l == l.max()).nonzero()[0]))
            probs.append(1.0)
            continue
        order = torch.argsort(l, descending=True, stable=True)
        w = torch.exp((l[order] - l.max()) / min(t, 2.0 ** 100))
        n = min(V, k) if k > 0 else V
        if not p >= 1.0:
            before = w[:n].cumsum(0) - w[:n]
            n = max(1, int((before < p * w[:n].sum()).sum())) if p > 0 else 1
        n = max(1, int((w[:n] >= low).sum())) if low > 0 else n
        keep, at = torch.sort(order[:n])
        w = w[:n][at]
        r = 0.0 if not r > 0 else r
        over = w.cumsum(0) > r * w.sum()
        i = int(over.nonzero()[0]) if bool(over.any()) else int((w > 0).nonzero()[-1])
        ids.append(int(keep[i]))
        probs.append(float(w[i] / w.sum()))
    return torch.tensor(ids, dtype=torch.int32), torch.tensor(probs, dtype=torch.float64)


def check(logits, u, **kw):
    es = _es()
    B = logits.shape[0]
    prob = torch.full((B,), 5.0, device="cuda")
    ids = es.sample_tokens(logits, u, prob=prob, **kw)
    wi, wp = want(logits, u, **kw)
    assert torch.equal(ids.cpu(), wi), (ids.cpu().tolist(), wi.tolist())
    p = prob.double().cpu()
    assert torch.equal(p.isnan(), wp.isnan())
    assert bool(((p - wp).abs() <= wp * 2.0 ** -23)[~wp.isnan()].all()), (p, wp)
    assert torch.equal(es.sample_tokens(logits, u, **kw), ids)
    return ids


def rows(B, V, seed=0, std=3.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, V, generator=g) * std).to(dtype).cuda(), torch.rand(B, generator=g).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 2049, 50257, 131072])
@pytest.mark.parametrize("kw", [{}, dict(temperature=0.7), dict(top_k=1), dict(top_k=40), dict(top_p=0.9), dict(min_p=0.05),
                                dict(temperature=1.7, top_k=300, top_p=0.8, min_p=0.01), dict(top_k=10 ** 9, top_p=0.999),
                                dict(temperature=0.0)])
def test_choices(dtype, V, kw):
    l, u = rows(7, V, seed=V % 1000 + len(kw), dtype=dtype)
    check(l, u, **kw)


@pytest.mark.parametrize("B,V", [(1, 393216), (200, 5000), (33, 32001)])
def test_sizes(B, V):
    l, u = rows(B, V, seed=B)
    check(l, u, temperature=0.9, top_p=0.95)
    check(l, u, top_k=V // 2, min_p=1e-6)


def test_choices_of_each_row():
    l, u = rows(24, 3001, seed=5, dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(6)
    t = torch.rand(24, generator=g) * 2
    t[::5] = 0.0
    k = torch.randint(0, 60, (24,), generator=g).to(torch.int32)
    p = (torch.rand(24, generator=g) * 1.2).float()
    m = (torch.rand(24, generator=g) * 0.3 * (torch.arange(24) % 2)).float()
    check(l, u, temperature=t.cuda(), top_k=k.cuda(), top_p=p.cuda(), min_p=m.cuda())
    check(l, u, temperature=t.cuda(), top_p=0.7)


def test_ties():
    """Equal logits: the cut keeps the lowest indices."""
    l = torch.zeros(8, 5000, device="cuda")
    u = torch.tensor([0.0, 0.1, 0.25, 0.5, 0.75, 0.9, 0.999, 1.0 - 2.0 ** -24], device="cuda")
    for kw in (dict(), dict(top_k=7), dict(top_k=4999), dict(top_p=0.5), dict(top_p=1e-9), dict(top_k=1000, top_p=0.25),
               dict(min_p=1.0), dict(min_p=0.999)):
        check(l, u, **kw)
    # three levels, the cut inside the middle one, which is spread over the row
    l = (torch.arange(5000) * 7919 % 3).float().cuda().repeat(8, 1)
    for kw in (dict(top_k=1667), dict(top_k=2000), dict(top_k=3333), dict(top_p=0.8), dict(top_p=0.95), dict(top_k=2500, top_p=0.9)):
        check(l, u, **kw)
    # two equal halves: the border itself belongs to the second
    l = torch.zeros(2, 2, device="cuda")
    u = torch.tensor([0.5, 0.5 - 2.0 ** -25], device="cuda")
    assert check(l, u).tolist() == [1, 0]
    # zeros of either sign are equal
    l = torch.tensor([[-0.0, 0.0, -0.0, -1.0]], device="cuda")
    assert check(l, u[1:], top_k=1).tolist() == [0]
    assert check(l, u[:1], temperature=0.0).tolist() == [0]


def test_masked_and_non_finite_rows():
    inf, nan = float("inf"), float("nan")
    l, u = rows(10, 700, seed=2)
    l[0] = -inf
    l[1, 1:] = -inf
    l[2, :699] = -inf
    l[3, 5] = nan
    l[4, 6] = inf
    l[5, ::2] = -inf
    l[6] = torch.finfo(torch.float32).min
    l[7, 10:] = torch.finfo(torch.float32).min
    l[8, 3] = torch.finfo(torch.float32).max
    l[9, :350] = -inf
    for kw in (dict(), dict(top_k=5), dict(top_p=0.9), dict(top_k=400, top_p=0.5, min_p=0.01), dict(temperature=0.0),
               dict(temperature=100.0), dict(temperature=1e-3)):
        ids = check(l, u, **kw).tolist()
        assert ids[0] == ids[3] == ids[4] == -1 and ids[1] == 0 and ids[2] == 699
    # values whose pattern is near that of the largest, and far from 0
    l = torch.full((1, 3000), 1e30, device="cuda") * (1 + torch.arange(3000, device="cuda") % 7 * 2.0 ** -22)
    check(l, u[:1], top_k=1500, temperature=1e24)


@pytest.mark.parametrize("std", [1e-30, 1e-6, 1e-2, 30.0, 1e4])
def test_spreads(std):
    """Logits in a narrow or a wide range: the bins' widths follow."""
    l, u = rows(6, 9000, seed=3, std=std)
    for kw in (dict(), dict(top_k=100), dict(top_p=0.6), dict(top_k=5000, top_p=0.5)):
        check(l, u, **kw)
    check(l, u, top_k=50, top_p=0.7, temperature=std)
    # a few far above the rest, which then lie in one bin
    l[:, 77] += 100 * std
    l[:, 8999] -= 1000 * std
    check(l, u, top_k=200, temperature=std)
    check(l, u, top_p=0.5, temperature=50 * std)


def test_extreme_arguments():
    l, u = rows(6, 4000, seed=8)
    nan, inf = float("nan"), float("inf")
    u = torch.tensor([0.0, -1.0, nan, 1.0 - 2.0 ** -24, 1e-30, 0.5], device="cuda")
    for kw in (dict(), dict(top_p=0.0), dict(top_p=-1.0), dict(top_p=nan), dict(top_p=inf), dict(min_p=nan), dict(min_p=-1.0),
               dict(min_p=2.0), dict(top_k=-5), dict(temperature=nan), dict(temperature=-2.0), dict(temperature=inf),
               dict(temperature=1e38), dict(temperature=1e-25), dict(temperature=1e-35), dict(min_p=1e-38)):
        check(l, u, **kw)
    # u of 1 and above: the last kept token
    u = torch.tensor([1.0, 2.0, inf, 1.0, 1.0, 1.0], device="cuda")
    ids = _es().sample_tokens(l, u, top_k=9)
    keep = torch.topk(l, 9, 1).indices.max(1).values
    assert torch.equal(ids.long(), keep)


@pytest.mark.parametrize("dtype,ld,off", [(torch.bfloat16, 1003, 1), (torch.float32, 1001, 3), (torch.float16, 1008, 8), (torch.float32, 1000, 0)])
def test_strides(dtype, ld, off):
    l, u = rows(5, 1000, seed=9, dtype=dtype)
    wide = torch.full((5 * ld + off + 8,), float("nan"), dtype=dtype, device="cuda")
    view = wide[off:off + 5 * ld].view(5, ld)[:, :1000]
    view.copy_(l)
    ids = check(view, u, top_p=0.9)
    assert torch.equal(ids, _es().sample_tokens(l, u, top_p=0.9))


def test_shares():
    """20000 random numbers over one row: each token's share of them is its probability, within five standard deviations."""
    V, n = 50, 20000
    l, _ = rows(1, V, seed=4, std=1.0)
    u = (torch.arange(n, dtype=torch.float64) + 0.5).div(n).float().cuda()
    ids = _es().sample_tokens(l.expand(n, V), u, temperature=0.8)
    share = torch.bincount(ids.long(), minlength=V).double() / n
    # equidistant numbers: each share is off by one of them at most
    assert bool(((share - torch.softmax(l[0].double() / 0.8, 0)).abs() <= 1.01 / n).all())


def test_capture_and_streams():
    es = _es()
    l, u = rows(9, 32000, seed=7)
    ids = torch.zeros(9, dtype=torch.int32, device="cuda")
    es.sample_tokens(l, u, top_k=50, top_p=0.9, out=ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        es.sample_tokens(l, u, top_k=50, top_p=0.9, out=ids)
    for seed in range(3):
        l2, u2 = rows(9, 32000, seed=20 + seed)
        l.copy_(l2)
        u.copy_(u2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids.cpu(), want(l, u, top_k=50, top_p=0.9)[0])
    outs = []
    for st in [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(st):
            outs += [es.sample_tokens(l, u, top_k=50, top_p=0.9) for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ids) for o in outs)


def test_refusals():
    es = _es()
    l, u = rows(3, 100)
    ok = dict(logits=l, u=u)
    for kw in (dict(logits=l.double()), dict(logits=l.cpu()), dict(logits=l[0]), dict(logits=l.t()), dict(logits=l[:, :0]),
               dict(u=u[:2]), dict(u=u.double()), dict(u=0.5), dict(u=u.cpu()), dict(temperature=u[:1]),
               dict(top_k=u), dict(top_p=u.double()), dict(min_p=u.cpu()), dict(out=torch.zeros(3, device="cuda")),
               dict(out=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(prob=u[:2])):
        with pytest.raises(ValueError):
            es.sample_tokens(**{**ok, **kw})
    with pytest.raises(ValueError):
        es.sample_tokens(torch.zeros(1, es.SAMPLE_MAX_V + 1, device="cuda"), u[:1])
    assert es.sample_tokens(l[:0], u[:0]).shape == (0,)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kw", [dict(top_k=1500, temperature=2.0), dict(top_p=0.97, temperature=3.0), dict(top_k=20000, top_p=0.9),
                                dict(top_p=0.3, temperature=0.2), dict(top_k=1024), dict(top_k=1025), dict(temperature=50.0, top_p=0.5)])
def test_large_sets(dtype, kw):
    """More kept tokens than one CTA sorts, at its limit and past it; cuts in the bulk of 60000 tokens."""
    l, u = rows(5, 60000, seed=11, std=2.5, dtype=dtype)
    check(l, u, **kw)


def test_many_equal_values():
    """More equal logits at the cut than one CTA sorts, spread over the row or together."""
    for l in ((torch.arange(40000) * 7919 % 5).float().repeat(3, 1).cuda(), (torch.arange(40000) // 9000).float().repeat(3, 1).cuda()):
        u = torch.tensor([0.01, 0.5, 0.99], device="cuda")
        for kw in (dict(top_k=5000), dict(top_k=12345, top_p=0.9), dict(top_p=0.5), dict(top_p=0.99, temperature=0.3)):
            check(l, u, **kw)


@pytest.mark.parametrize("B", [1, 3, 20, 80, 160, 700])
def test_rows_and_ctas(B):
    """Rows that have eight, four, two CTAs and one, with and without cuts."""
    l, u = rows(B, 9001, seed=B)
    check(l, u)
    check(l, u, min_p=0.05, temperature=0.8)
    check(l, u, top_k=30, top_p=0.9)
