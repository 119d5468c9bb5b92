"""Keys and values of new tokens into a paged cache, keys and queries rotated by position.

Tolerances: a rotated value is a cos - b sin. The angle is off by at most 2^-24 pi (its last 24 bits) + 2^-32 turns +
2^-53 position inv_freq, the sine and cosine by 2^-22, each product and the sum by 2^-24: together below 2^-20 of |a| + |b|
for positions below 2^30. Stored and returned values are rounded once more, by half a step (E4M3: 2^-4, or 2^-10
below its normal range, of the value times fl(1 / scale), which is off by 2^-23)."""
import pytest
import torch

from tests import _kv

pytestmark = pytest.mark.gpu


def _es():
    from routed_expert_ffn_topk_gb300 import estream as es
    return es


class _Step:
    """T tokens at the given positions of B sequences, their rows cut out of one projection's result."""

    def __init__(self, positions, rows, heads, Hq, dim, page, kind, x="bf16", by_head=False, scales=(1.0, 1.0), pad=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        T, B = len(positions), max(rows) + 1
        M = max(positions) // page + 1
        self.n = B * 3 + 2
        need = {(r, p // page) for r, p in zip(rows, positions) if p >= 0}
        ids = torch.randperm(len(need) + 2, generator=g).tolist()
        self.n = len(ids)
        table = torch.full((B, M), -1, dtype=torch.int32)
        for i, (r, e) in enumerate(sorted(need)):
            table[r, e] = ids[i]
        self.k, self.v = _kv.pages(self.n, page, heads, dim, kind, by_head, 3.0), _kv.pages(self.n, page, heads, dim, kind, by_head, 3.0)
        qkv = torch.randn(T, Hq + 2 * heads, dim + pad, generator=g).to(_kv.DT[x]).cuda()[..., pad:]
        self.q, self.nk, self.nv = qkv[:, :Hq], qkv[:, Hq:Hq + heads], qkv[:, Hq + heads:]
        self.table = table.cuda()
        self.positions = torch.tensor(positions, dtype=torch.int32).cuda()
        self.rows = torch.tensor(rows, dtype=torch.int32).cuda()
        self.pos_list, self.row_list, self.page, self.scales = positions, rows, page, scales
        self.cache = _es().PagedKV(self.k, self.v, *scales)

    def check(self, inv_freq, interleaved, q_out):
        pos = torch.tensor([max(p, 0) for p in self.pos_list]).cuda()
        f = inv_freq if inv_freq is not None else torch.zeros(0, device="cuda")
        want_k = torch.full(self.k.shape, 3.0, dtype=torch.float64, device="cuda")
        want_v, tol_k, tol_v = want_k.clone(), torch.zeros_like(want_k), torch.zeros_like(want_k)
        rk, sk = _kv.rotate64(self.nk.double(), pos, f, interleaved)
        rq, sq = _kv.rotate64(self.q.double(), pos, f, interleaved)
        t = [i for i, p in enumerate(self.pos_list) if p >= 0]
        page = torch.tensor([int(self.table[self.row_list[i], self.pos_list[i] // self.page]) for i in t]).cuda()
        slot = torch.tensor([self.pos_list[i] % self.page for i in t]).cuda()
        for want, tol, r, s, scale in ((want_k, tol_k, rk, sk, self.scales[0]),
                                       (want_v, tol_v, self.nv.double(), torch.zeros_like(rk), self.scales[1])):
            y = r[t] / scale
            slack = s[t] * 2.0 ** -20 / scale
            if self.k.dtype == torch.float8_e4m3fn:
                tol[page, slot] = (y.abs() + slack) * (2.0 ** -4 + 2.0 ** -22) + slack + 2.0 ** -10
                y = y.clamp(-448.0, 448.0)
            else:
                u = torch.finfo(self.k.dtype).eps / 2
                tol[page, slot] = (y.abs() + slack) * u + slack + 2.0 ** -25
            want[page, slot] = y
        dk, dv = (self.k.float().double() - want_k).abs(), (self.v.float().double() - want_v).abs()
        assert bool((dk <= tol_k).all()), float((dk - tol_k).max())
        assert bool((dv <= tol_v).all()), float((dv - tol_v).max())
        if q_out is not None:
            u = torch.finfo(q_out.dtype).eps / 2
            d = (q_out.double() - rq)[t].abs()
            assert bool((d <= (rq[t].abs() + sq[t] * 2.0 ** -20) * u + sq[t] * 2.0 ** -20 + 2.0 ** -25).all()), float(d.max())


def _inv(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().cuda()


@pytest.mark.parametrize("kind,x", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("dim,rot", [(16, 16), (64, 64), (80, 80), (128, 128), (128, 64), (128, 2), (96, 6), (256, 256), (64, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(kind, x, dim, rot, interleaved):
    s = _Step([0, 1, 17, 4095, 131071], [0, 1, 2, 3, 4], 2, 6, dim, 16, kind, x, seed=dim + rot,
              scales=(0.02, 1.5) if kind == "e4m3" else (1.0, 1.0))
    f = _inv(rot) if rot else None
    q = _es().kv_append(s.cache, s.nk, s.nv, s.positions, s.table, q=s.q, inv_freq=f, interleaved=interleaved)
    s.check(f, interleaved, q)


@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("by_head", [False, True])
@pytest.mark.parametrize("pad", [0, 1])
def test_prompts(page, by_head, pad):
    """Whole prompts, rows named by index, padding behind them; pad 1: rows that start on odd elements."""
    pos, rows = [], []
    for r, n in enumerate((1, 40, 133)):
        pos += list(range(n))
        rows += [r] * n
    pos += [-1, -1, -5]
    rows += [0, 2, 1]
    s = _Step(pos, rows, 3, 4, 64, page, "bf16", by_head=by_head, pad=pad)
    q_out = torch.full(s.q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    f = _inv(64)
    got = _es().kv_append(s.cache, s.nk, s.nv, s.positions, s.table, rows=s.rows, q=s.q, q_out=q_out, inv_freq=f)
    assert got is q_out
    s.check(f, False, q_out)
    assert bool((q_out[-3:] == 9.0).all())  # padding leaves its rows


def test_many_tokens():
    """More tokens than blocks of a launch, every fourth of them padding."""
    n = 6000
    s = _Step([i if i % 4 else -1 for i in range(n)], [0] * n, 1, 2, 32, 16, "bf16")
    f = _inv(32)
    q_out = torch.full(s.q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    _es().kv_append(s.cache, s.nk, s.nv, s.positions, s.table, rows=s.rows, q=s.q, q_out=q_out, inv_freq=f)
    s.check(f, False, q_out)
    assert bool((q_out[::4] == 9.0).all())


def test_keys_alone_and_in_place():
    s = _Step([5, 6, 7], [0, 0, 1], 2, 4, 64, 16, "f16", "f16")
    f = _inv(64)
    before = s.q.clone()
    assert _es().kv_append(s.cache, s.nk, s.nv, s.positions, s.table, rows=s.rows, inv_freq=f) is None
    s.check(f, False, None)
    assert torch.equal(s.q, before)
    out = _es().kv_append(s.cache, s.nk, s.nv, s.positions, s.table, rows=s.rows, q=s.q, inv_freq=f)
    _es().kv_append(s.cache, s.nk, s.nv, s.positions, s.table, rows=s.rows, q=s.q, q_out=s.q, inv_freq=f)
    assert torch.equal(s.q, out)
    s.q.copy_(before)


def test_far_positions():
    """2^30 positions: the angle keeps its place in the turn."""
    es = _es()
    far = 1 << 30
    k, v = _kv.pages(1, 64, 1, 64, "f16"), _kv.pages(1, 64, 1, 64, "f16")
    x = torch.randn(4, 1, 64, generator=torch.Generator().manual_seed(0)).half().cuda()
    pos = torch.tensor([far - 1, far - 1001, far // 3, 12345679], dtype=torch.int32, device="cuda")
    table = torch.zeros(1, far // 64, dtype=torch.int32, device="cuda").expand(4, -1)
    f = _inv(64)
    q = es.kv_append(es.PagedKV(k, v), x, x, pos, table, q=x, inv_freq=f)
    want, size = _kv.rotate64(x.double(), pos, f, False)
    assert bool(((q.double() - want).abs() <= (want.abs() + size * 2.0 ** -20) * 2.0 ** -11 + size * 2.0 ** -20 + 2.0 ** -25).all())


def test_bad_places():
    """A token without a valid page is not stored and its queries are NaN; the others are."""
    es = _es()
    s = _Step([3, 20, 40, 9, 11], [0, 1, 2, 3, 4], 2, 4, 64, 16, "bf16")
    f = _inv(64)
    good = es.kv_append(s.cache, s.nk, s.nv, s.positions, s.table, q=s.q, inv_freq=f)
    kept = s.k.clone()
    s.k.fill_(3.0)
    s.v.fill_(3.0)
    pages = [int(s.table[i, p // 16]) for i, p in enumerate(s.pos_list)]
    s.table[1, 1] = -1
    s.table[2, 2] = s.n
    s.positions[3] = 16 * s.table.shape[1]
    rows = s.rows.clone()
    rows[4] = 5
    got = es.kv_append(s.cache, s.nk, s.nv, s.positions, s.table, rows=rows, q=s.q, inv_freq=f)
    assert bool(got[1:].isnan().all()) and torch.equal(got[0], good[0])
    assert torch.equal(s.k[pages[0]], kept[pages[0]])
    s.k[pages[0]], s.v[pages[0]] = 3.0, 3.0
    assert bool((s.k == 3.0).all()) and bool((s.v == 3.0).all())
    rows[4] = -1
    assert bool(es.kv_append(s.cache, s.nk, s.nv, s.positions, s.table, rows=rows, q=s.q, inv_freq=f)[4].isnan().all())


def test_e4m3_limits():
    """Values past 448 scales are the largest, NaN stays NaN."""
    es = _es()
    k = _kv.pages(1, 1, 1, 16, "e4m3", fill=0.0)
    v = k.clone()
    x = torch.tensor([[[1000.0, -1000.0, float("inf"), float("-inf"), float("nan"), 448.0, 460.0, 0.0] * 2]], device="cuda").half()
    es.kv_append(es.PagedKV(k, v), x, x, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    want = torch.tensor([448.0, -448.0, 448.0, -448.0, float("nan"), 448.0, 448.0, 0.0] * 2)
    for t in (k, v):
        assert torch.equal(t.float().cpu().view(-1).nan_to_num(7.0), want.nan_to_num(7.0))


def test_append_then_attend():
    """A prompt and then tokens one by one, each appended and at once attended to, in one captured graph: the rows
    of a causal mask over rotated keys, within the bounds of both calls."""
    es = _es()
    n, heads, Hq, D, page = 60, 2, 6, 64, 16
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn(2, n, Hq + 2 * heads, D, generator=g).bfloat16().cuda()
    f = _inv(D)
    k, v = _kv.pages(2 * 4 + 1, page, heads, D, "bf16"), _kv.pages(2 * 4 + 1, page, heads, D, "bf16")
    cache = es.PagedKV(k, v)
    table = (torch.randperm(8, generator=g) + 1).view(2, 4).to(torch.int32).cuda()
    m = 37
    pos = torch.arange(m, dtype=torch.int32).repeat(2).cuda()
    rows = torch.arange(2, dtype=torch.int32).repeat_interleave(m).cuda()
    first = qkv[:, :m].reshape(2 * m, -1, D)
    q = es.kv_append(cache, first[:, Hq:Hq + heads], first[:, Hq + heads:], pos, table, rows=rows, q=first[:, :Hq], inv_freq=f)
    got = [es.kv_attend(cache, q, table[rows.long()], pos + 1).view(2, m, Hq, D)]
    now, at, out = qkv[:, m].clone(), torch.full((2,), m, dtype=torch.int32, device="cuda"), torch.zeros(2, Hq, D, dtype=torch.bfloat16, device="cuda")

    def step():
        q = es.kv_append(cache, now[:, Hq:Hq + heads], now[:, Hq + heads:], at, table, q=now[:, :Hq], inv_freq=f)
        es.kv_attend(cache, q, table, at + 1, out=out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(m, n):
        now.copy_(qkv[:, i])
        at.fill_(i)
        graph.replay()
        got.append(out.clone()[:, None])
    got = torch.cat(got, 1).double().cpu()
    whole = torch.arange(n).cuda()
    for b in range(2):
        rq, _ = _kv.rotate64(qkv[b, :, :Hq].double(), whole, f, False)
        rk, _ = _kv.rotate64(qkv[b, :, Hq:Hq + heads].double(), whole, f, False)
        for h in range(Hq):
            kk, vv = rk[:, h // 3], qkv[b, :, Hq + heads + h // 3].double()
            z = (rq[:, h] @ kk.t()) * D ** -0.5
            z = z.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), float("-inf"))
            w = torch.softmax(z, 1)
            want, mean = (w @ vv).cpu(), (w @ vv.abs()).cpu()
            # query and key are rounded to bf16 (2^-8 each) before they meet: scores off by 2^-7 of their size
            size = float((rq[:, h].abs() @ kk.abs().t()).max()) * D ** -0.5
            tol = mean * 2 * (2.0 ** -7 * size) * 1.1 + 2.0 ** -8 * want.abs() + mean * 2.0 ** -12
            assert bool(((got[b, :, h] - want).abs() <= tol).all())


def test_refusals():
    es = _es()
    s = _Step([3, 20], [0, 1], 2, 4, 64, 16, "bf16")
    f = _inv(64)
    good = dict(k=s.nk, v=s.nv, positions=s.positions, table=s.table, q=s.q, inv_freq=f)
    for kw in (dict(k=s.nk[:, :1]), dict(k=s.nk.half()), dict(k=s.nk.float()), dict(v=s.nv[:1]), dict(v=s.nv[..., :32]),
               dict(v=s.nv.half()), dict(q=s.q.half()), dict(q=s.q[:1]), dict(positions=s.positions.long()),
               dict(positions=s.positions[:1]), dict(table=s.table.long()), dict(table=s.table[:1]), dict(rows=s.rows[:1]),
               dict(rows=s.rows.long()), dict(inv_freq=f.double()), dict(inv_freq=torch.ones(33, device="cuda")),
               dict(inv_freq=f.cpu()), dict(q=None, q_out=s.q), dict(q_out=s.q.half()), dict(k=s.nk.cpu())):
        with pytest.raises(ValueError):
            es.kv_append(s.cache, **{**good, **kw})
    assert es.kv_append(s.cache, s.nk[:0], s.nv[:0], s.positions[:0], s.table) is None


@pytest.mark.parametrize("size", [0.0, 2.0 ** -140, 1e-8, 0.999, 1.0, 1.999, 2.0, 7.25, 1000.5])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_frequencies_of_any_size(size, sign):
    """Slow, fast and negative turns; below 2 they are formed in integers, from there in 64 bits."""
    s = _Step([0, 1, 999, 65537], [0, 1, 2, 3], 1, 2, 32, 16, "f16", "f16")
    f = torch.full((16,), sign * size).cuda() * torch.linspace(0.5, 1.0, 16).cuda()
    q = _es().kv_append(s.cache, s.nk, s.nv, s.positions, s.table, q=s.q, inv_freq=f)
    s.check(f, False, q)


@pytest.mark.parametrize("heads,Hq,dim", [(1, 0, 16), (1, 1, 256), (7, 49, 64), (64, 64, 128), (3, 300, 48)])
@pytest.mark.parametrize("T", [1, 3, 400])
def test_head_counts(heads, Hq, dim, T):
    """Few and many heads, over few warps and many."""
    s = _Step(list(range(T)), [0] * T, heads, Hq, dim, 16, "bf16")
    f = _inv(dim)
    q = _es().kv_append(s.cache, s.nk, s.nv, s.positions, s.table, rows=s.rows, q=s.q if Hq else None, inv_freq=f)
    s.check(f, False, q)
