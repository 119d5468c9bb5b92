"""Attention of one new token per row over a paged cache, against its formula in 64 bits; tolerances are those
that tests/_kv.py derives. The cache holds NaN wherever a call has no business."""
import math

import pytest
import torch

from tests import _kv

pytestmark = pytest.mark.gpu


def _es():
    from routed_expert_ffn_topk_gb300 import estream as es
    return es


def _q(B, Hq, D, kind, seed=1, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, Hq, D, generator=g) * std).to(_kv.DT[kind]).cuda()


def _check(c, q, scale=None, **kw):
    es = _es()
    out = torch.full(q.shape, 7.0, device="cuda").to(q.dtype)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    got = es.kv_attend(c.cache, q, c.table, c.lens, scale=scale, window=c.window, out=out, lse=lse, **kw)
    assert got is out
    want, wl, tol, ltol = c.want(q, q.shape[2] ** -0.5 if scale is None else scale)
    y, l = out.double().cpu(), lse.double().cpu()
    empty = torch.tensor(c.lens_list) == 0
    assert torch.equal(y[empty], torch.zeros_like(y[empty])) and bool((l[empty] == -math.inf).all())
    d = (y - want).abs()
    assert bool((d <= tol).all()), (float((d / tol.clamp(min=1e-30)).max()), float(d.max()))
    dl = (l - wl)[~empty].abs()
    assert bool((dl <= ltol[~empty]).all()), float(dl.max())
    return out, lse


@pytest.mark.parametrize("kind,qk", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 128, 160, 256])
@pytest.mark.parametrize("page", [1, 7, 16, 48])
def test_types_and_widths(kind, qk, dim, page):
    c = _kv.Case([0, 1, 15, 16, 17, 64, 65, 130, 333], 2, dim, page, kind, seed=dim + page,
                 scales=(0.25, 3.0) if kind == "e4m3" else (1.0, 1.0))
    _check(c, _q(9, 6, dim, qk))


@pytest.mark.parametrize("heads,group", [(1, 1), (1, 8), (2, 9), (3, 16), (1, 17), (2, 33), (16, 1), (5, 4)])
@pytest.mark.parametrize("by_head", [False, True])
def test_head_layouts(heads, group, by_head):
    c = _kv.Case([200, 1, 0, 77], heads, 64, 16, "bf16", by_head=by_head, seed=heads)
    _check(c, _q(4, heads * group, 64, "bf16"))


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("lens,heads", [([20000], 2), ([5000, 3], 1), ([1, 9000, 0, 0, 2, 4097], 4), ([30] * 300, 3),
                                        ([0] * 5 + [100] + [0] * 7, 2), ([0, 0], 1)])
def test_split_over_the_length(kind, lens, heads):
    c = _kv.Case(lens, heads, 128, 32, kind, seed=len(lens))
    out, lse = _check(c, _q(len(lens), 4 * heads, 128, "bf16" if kind == "e4m3" else kind))
    again, _ = _check(c, _q(len(lens), 4 * heads, 128, "bf16" if kind == "e4m3" else kind))
    assert torch.equal(out, again)  # bit for bit


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 4096, 1 << 30])
@pytest.mark.parametrize("page", [5, 16])
def test_window(window, page):
    c = _kv.Case([0, 1, 16, 17, 100, 101, 2500], 2, 64, page, "f16", window=window, seed=window % 97)
    # pages wholly before the window are gone
    for b, n in enumerate(c.lens_list):
        c.table[b, :max(0, n - window) // page] = -1
    _check(c, _q(7, 4, 64, "f16"))


@pytest.mark.parametrize("scale", [0.0, -0.7, 3.0])
def test_scale(scale):
    _check(_kv.Case([40, 700], 1, 32, 16, "bf16"), _q(2, 3, 32, "bf16"), scale=scale)


def test_strides():
    """Queries out of a wider buffer that starts on an odd element, results into another, the table's rows apart."""
    es = _es()
    c = _kv.Case([33, 500, 0], 2, 80, 16, "bf16")
    q = _q(3, 6, 80, "bf16")
    wide = torch.zeros(3 * 7 * 91 + 1, dtype=q.dtype, device="cuda")[1:].view(3, 7, 91)[:, :6, :80]
    wide.copy_(q)
    whole = torch.full((3, 8, 100), 5.0, dtype=q.dtype, device="cuda")
    out = whole[:, 1:7, 3:83]
    table = torch.full((3, c.table.shape[1] + 9), 12345, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    es.kv_attend(c.cache, wide, table[:, :c.table.shape[1]], c.lens, out=out)
    want = es.kv_attend(c.cache, q, c.table, c.lens)
    assert torch.equal(out, want)
    whole[:, 1:7, 3:83] = 5.0
    assert bool((whole == 5.0).all())
    # in place
    es.kv_attend(c.cache, q, c.table, c.lens, out=q)
    assert torch.equal(q, want)


def test_rows_of_one_sequence():
    """The tokens of a prompt: rows of one table row, each with its own length, give the rows of a causal mask."""
    n = 150
    c = _kv.Case([n], 2, 64, 16, "bf16")
    q = _q(n, 4, 64, "bf16")
    lens = torch.arange(1, n + 1, dtype=torch.int32, device="cuda")
    got = _es().kv_attend(c.cache, q, c.table.expand(n, -1), lens)
    for i in (0, 1, 15, 16, 70, n - 1):
        one = _es().kv_attend(c.cache, q[i:i + 1], c.table, lens[i:i + 1])
        want, _, tol, _ = _one(c, q[i:i + 1], i + 1)
        assert bool(((got[i].double().cpu() - want[0]).abs() <= tol[0]).all()), i
        assert bool(((one[0].double().cpu() - want[0]).abs() <= tol[0]).all()), i


def _one(c, q, n):
    p, s = c.place[0]
    keep, c.place = c.place, [(p[:n], s[:n])]
    try:
        return c.want(q, q.shape[2] ** -0.5)
    finally:
        c.place = keep


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_bad_pages_and_lengths(kind):
    """A needed page or a length out of range makes its row NaN and leaves the others."""
    es = _es()
    lens = [100, 100, 100, 100, 100, 100, 100]
    c = _kv.Case(lens, 2, 64, 16, kind)
    q = _q(7, 4, 64, "bf16")
    good = es.kv_attend(c.cache, q, c.table, c.lens)
    c.table[1, 0] = -1
    c.table[2, 6] = c.k.shape[0]
    c.table[3, 3] = 2 ** 31 - 1
    c.lens[4] = -1
    c.lens[5] = 7 * 16 + 1
    lse = torch.zeros(7, 4, device="cuda")
    got = es.kv_attend(c.cache, q, c.table, c.lens, lse=lse)
    assert bool(got[1:6].isnan().all()) and bool(lse[1:6].isnan().all())
    assert torch.equal(got[[0, 6]], good[[0, 6]]) and bool(lse[[0, 6]].isfinite().all())


def test_no_pages():
    es = _es()
    k = torch.empty(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache = es.PagedKV(k, k)
    q = _q(2, 4, 64, "bf16")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    for M in (0, 3):
        table = torch.zeros(2, M, dtype=torch.int32, device="cuda")
        assert bool((es.kv_attend(cache, q, table, lens) == 0).all())
        assert bool(es.kv_attend(cache, q, table, lens + 1).isnan().all())
    assert es.kv_attend(cache, q[:0], torch.zeros(0, 3, dtype=torch.int32, device="cuda"), lens[:0]).shape == (0, 4, 64)


def test_infinite_and_large_values():
    """Scores of -infinity weigh nothing; a NaN key makes the heads that meet it NaN; large values stay finite."""
    es = _es()
    c = _kv.Case([50, 50, 50, 50], 2, 64, 16, "bf16")
    q = _q(4, 4, 64, "bf16").abs()
    p, s = c.place[0]
    c.k[p[3], s[3], 0] = float("-inf")
    c.k[c.place[1][0], c.place[1][1]] = float("-inf")
    c.k[c.place[2][0][7], c.place[2][1][7], 1, 5] = float("nan")
    c.v[c.place[3][0], c.place[3][1]] *= 2.0 ** 100
    lse = torch.zeros(4, 4, device="cuda")
    out = es.kv_attend(c.cache, q, c.table, c.lens, lse=lse)
    c.place[0] = (torch.cat([p[:3], p[4:]]), torch.cat([s[:3], s[4:]]))
    c.place[1] = c.place[2] = (p[:0], s[:0])
    want, wl, tol, _ = c.want(q, 0.125)
    assert bool(((out.double().cpu() - want)[0, :2].abs() <= tol[0, :2]).all())
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())
    assert bool(out[2, 2:].isnan().all()) and bool(out[2, :2].isfinite().all())
    assert bool(((out.double().cpu() - want)[3].abs() <= tol[3]).all())


def test_far_scores():
    """One score far above the others, at either end; and all scores far from zero."""
    for at in (0, 299):
        c = _kv.Case([300], 1, 64, 16, "f16")
        p, s = c.place[0]
        q = _q(1, 2, 64, "f16")
        c.k[p[at], s[at], 0] = (q[0, 0].float() * 4).half()
        _check(c, q, scale=1.0)
    c = _kv.Case([300], 1, 64, 16, "bf16")
    p, s = c.place[0]
    c.k[p, s] += 20.0
    _check(c, torch.full((1, 2, 64), 8.0, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("std", [2.0 ** -120, 2.0 ** -20, 2.0 ** 60])
def test_e4m3_queries_of_any_size(std):
    """Next to an 8-bit cache queries are scaled by a power of two before they are multiplied."""
    c = _kv.Case([90, 1], 2, 64, 16, "e4m3", scales=(0.5, 0.5))
    q = _q(2, 4, 64, "bf16", std=std)
    _check(c, q, scale=min(1.0, 0.2 / std) if std > 1 else 1.0)


def test_offsets_past_32_bits():
    """Pages whose elements lie past 2^31 and whose bytes lie past 2^32."""
    page, heads, dim, total = 64, 64, 128, 8700  # 2^19 elements a page
    k = torch.empty(total, page, heads, dim, dtype=torch.bfloat16, device="cuda")
    es = _es()
    v = k
    table = torch.arange(total - 40, total, dtype=torch.int32, device="cuda")[None]
    k[total - 40:] = torch.randn(40, page, heads, dim, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16()
    q = _q(1, heads, dim, "bf16")
    lens = torch.tensor([40 * page - 5], dtype=torch.int32, device="cuda")
    got = es.kv_attend(es.PagedKV(k, v), q, table, lens)
    low = k[total - 40:].clone()
    want = es.kv_attend(es.PagedKV(low, low), q, table - (total - 40), lens)
    assert torch.equal(got, want) and bool(got.isfinite().all())


def test_streams_and_graphs():
    """Two streams at once with workspaces of their own, and a captured graph whose lengths grow between replays."""
    es = _es()
    c = _kv.Case([3000, 100, 0, 2000], 2, 128, 16, "bf16")
    q = _q(4, 8, 128, "bf16")
    want = es.kv_attend(c.cache, q, c.table, c.lens)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    for _ in range(20):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(es.kv_attend(c.cache, q, c.table, c.lens))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    lens, out = c.lens.clone(), torch.zeros_like(q)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        es.kv_attend(c.cache, q, c.table, lens, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        es.kv_attend(c.cache, q, c.table, lens, out=out)
    for cut in (0, 1, 50, 99):
        lens.copy_((c.lens - cut).clamp(min=0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, es.kv_attend(c.cache, q, c.table, lens)), cut


def test_workspace():
    """A given workspace holds anything before the call; one that is too small is refused."""
    es = _es()
    c = _kv.Case([30000, 100], 2, 64, 16, "bf16")
    q = _q(2, 8, 64, "bf16")
    want = es.kv_attend(c.cache, q, c.table, c.lens)
    n = c.cache.attend_workspace_bytes(2, 8, c.table.shape[1])
    assert n > 0
    for byte in (0, 0x7f, 0xff):
        ws = torch.full((n,), byte, dtype=torch.uint8, device="cuda")
        assert torch.equal(es.kv_attend(c.cache, q, c.table, c.lens, workspace=ws), want)
    with pytest.raises(ValueError):
        es.kv_attend(c.cache, q, c.table, c.lens, workspace=ws[:-16])


def test_refusals():
    es = _es()
    c = _kv.Case([30, 10], 2, 64, 16, "bf16")
    q = _q(2, 4, 64, "bf16")
    for kw in (dict(q=q.half()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(q=q.cpu()), dict(q=q[0]),
               dict(lens=c.lens.long()), dict(lens=c.lens[:1]), dict(lens=c.lens.cpu()), dict(table=c.table.long()),
               dict(table=c.table[:1]), dict(table=c.table.t()), dict(window=-1), dict(out=q.float()), dict(out=q[:1]),
               dict(lse=torch.zeros(2, 4)), dict(lse=torch.zeros(2, 5, device="cuda"))):
        a = dict(q=q, table=c.table, lens=c.lens)
        a.update(kw)
        with pytest.raises(ValueError):
            es.kv_attend(c.cache, **a)
    with pytest.raises(es.EStreamError):
        es.kv_attend(c.cache, q, c.table, c.lens, scale=float("nan"))
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    for bad in ((k, k.half()), (k.float(), k.float()), (k[..., :40], k[..., :40]), (k, k[:2]), (k[0], k[0]),
                (k[..., 1:49], k[..., 1:49]), (k[:, :, :, ::2], k[:, :, :, ::2]), (k[:1].expand(4, 16, 2, 64),) * 2, (k.cpu(), k.cpu())):
        with pytest.raises(ValueError):
            es.PagedKV(*bad)
    for s in (0.5, 0.0, float("nan")):
        with pytest.raises(ValueError):
            es.PagedKV(k, k, s)


@pytest.mark.parametrize("B,heads,n", [(1, 1, 4097), (1, 8, 4096), (2, 16, 2048), (4, 16, 600), (40, 8, 100), (37, 1, 64), (300, 1, 33)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_units_and_clusters(B, heads, n, kind):
    """On both sides of the rule by which a unit gets a cluster of its own: lengths from nothing to the table's end."""
    g = torch.Generator().manual_seed(B + n)
    lens = torch.randint(0, n + 1, (B,), generator=g).tolist()
    lens[-1] = n
    c = _kv.Case(lens, heads, 64, 16, kind, M=-(-n // 16), seed=n)
    _check(c, _q(B, 2 * heads, 64, "bf16"))


def test_two_graphs_at_once():
    """Two captured graphs over one cache, replayed on two streams at once, with and without a workspace."""
    es = _es()
    for n in (500, 40000):
        c = _kv.Case([n, n // 3], 2, 64, 16, "bf16")
        q = [_q(2, 8, 64, "bf16", seed=s) for s in (1, 2)]
        want = [es.kv_attend(c.cache, x, c.table, c.lens) for x in q]
        outs, graphs = [torch.zeros_like(x) for x in q], []
        for x, o in zip(q, outs):
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                for _ in range(20):
                    es.kv_attend(c.cache, x, c.table, c.lens, out=o)
            graphs.append(graph)
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(5):
            for graph, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
