"""The compiled part of the binding next to the interpreted one: the same results for what both take, and
nothing taken that the interpreted one refuses."""
import pytest
import torch

from tests import _kv

pytestmark = pytest.mark.gpu


@pytest.fixture
def es():
    from routed_expert_ffn_topk_gb300 import estream
    estream.lib()
    assert estream._fast is not None
    return estream


def _both(monkeypatch, es, f):
    """f() by each way; the compiled one took the call."""
    taken = []

    class Fast:
        def __getattr__(self, name):
            def call(*a):
                st = getattr(real, name)(*a)
                taken.append(st)
                return st
            return call
    real = es._fast
    monkeypatch.setattr(es, "_fast", Fast())
    one = f()
    assert taken == [0], "the compiled way gave the call back"
    monkeypatch.setattr(es, "_fast", None)
    two = f()
    monkeypatch.setattr(es, "_fast", real)
    return one, two


@pytest.mark.parametrize("kind,x", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "f16")])
@pytest.mark.parametrize("views", [False, True])
def test_cache(monkeypatch, es, kind, x, views):
    g = torch.Generator(device="cuda").manual_seed(3)
    T, heads, Hq, dim, page = 5, 2, 6, 64, 16
    dt = _kv.DT[x]
    qkv = torch.randn(T, Hq + 2 * heads, dim, device="cuda", generator=g).to(dt)
    q, k, v = (qkv[:, a:b] if views else qkv[:, a:b].contiguous() for a, b in ((0, Hq), (Hq, Hq + heads), (Hq + heads, Hq + 2 * heads)))
    table = torch.randperm(12, device="cuda").to(torch.int32).reshape(3, 4)
    rows = torch.tensor([0, 2, 1, 1, 2], dtype=torch.int32, device="cuda")
    positions = torch.tensor([63, 0, 17, 18, -1], dtype=torch.int32, device="cuda")
    inv = 10000.0 ** (-torch.arange(0, 24, device="cuda").float() / 24)

    def append(interleaved):
        c = es.PagedKV(_kv.pages(12, page, heads, dim, kind), _kv.pages(12, page, heads, dim, kind))
        out = torch.zeros(T, Hq, dim, dtype=dt, device="cuda")
        es.kv_append(c, k, v, positions, table, rows=rows, q=q, inv_freq=inv, interleaved=interleaved, q_out=out)
        return out, c.k.view(torch.uint8).clone(), c.v.view(torch.uint8).clone()
    for interleaved in (False, True):
        for a, b in zip(*_both(monkeypatch, es, lambda: append(interleaved))):
            assert torch.equal(a, b)

    def plain():  # keys alone: neither rows, queries nor a rotation
        c = es.PagedKV(_kv.pages(12, page, heads, dim, kind), _kv.pages(12, page, heads, dim, kind))
        assert es.kv_append(c, k[:3], v[:3], positions[:3], table) is None
        return c.k.view(torch.uint8).clone(), c.v.view(torch.uint8).clone()
    for a, b in zip(*_both(monkeypatch, es, plain)):
        assert torch.equal(a, b)

    c = _kv.Case([3000, 0, 77], heads, dim, page, kind)
    qs, n = q[:3], c.cache.attend_workspace_bytes(3, Hq, c.table.shape[1])
    for scale, window in ((None, 0), (0.25, 50), (1, 0)):
        def attend():
            out, lse = torch.zeros(3, Hq, dim, dtype=dt, device="cuda"), torch.zeros(3, Hq, device="cuda")
            es.kv_attend(c.cache, qs, c.table, c.lens, scale, window, out=out, lse=lse,
                         workspace=torch.empty(n + 16, dtype=torch.uint8, device="cuda"))
            return out, lse
        for a, b in zip(*_both(monkeypatch, es, attend)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_sample(monkeypatch, es, dtype):
    g = torch.Generator(device="cuda").manual_seed(4)
    logits = (2 * torch.randn(6, 1003, device="cuda", generator=g)).to(dtype)
    u = torch.rand(6, device="cuda", generator=g)
    ks = torch.tensor([0, 1, 5, 2000, -3, 50], dtype=torch.int32, device="cuda")
    ps = torch.linspace(0.1, 1.0, 6, device="cuda")
    for kw in (dict(), dict(temperature=0), dict(temperature=0.7, top_k=40, top_p=0.9, min_p=0.01), dict(top_k=ks, top_p=ps),
               dict(temperature=ps, min_p=ps)):
        def call():
            out, prob = torch.full((6,), -7, dtype=torch.int32, device="cuda"), torch.zeros(6, device="cuda")
            es.sample_tokens(logits, u, **kw, out=out, prob=prob)
            return out, prob
        (a, pa), (b, pb) = _both(monkeypatch, es, call)
        assert torch.equal(a, b) and torch.equal(pa, pb)


def test_streams(es):
    """The current stream is the call's, also while it is captured."""
    c = _kv.Case([100, 20], 2, 64, 16, "bf16")
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    want = es.kv_attend(c.cache, q, c.table, c.lens)
    ws = torch.empty(c.cache.attend_workspace_bytes(2, 4, c.table.shape[1]) + 1, dtype=torch.uint8, device="cuda")
    logits, u = torch.randn(2, 500, device="cuda"), torch.rand(2, device="cuda")
    ids = es.sample_tokens(logits, u)
    side = torch.cuda.Stream()
    out, to = torch.zeros_like(q), torch.zeros_like(ids)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        es.kv_attend(c.cache, q, c.table, c.lens, out=out, workspace=ws)
        es.sample_tokens(logits, u, out=to)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(to, ids)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        es.kv_attend(c.cache, q, c.table, c.lens, out=out, workspace=ws)
        es.sample_tokens(logits, u, out=to)
    out.zero_(), to.fill_(-9)
    torch.cuda.synchronize()
    assert not out.any() and (to == -9).all()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(to, ids)


class Own(torch.Tensor):
    pass


def test_refusals(es):
    """With an out, where the compiled way is asked first."""
    c = _kv.Case([30000, 10], 2, 64, 16, "bf16")
    q, lse = torch.zeros(2, 4, 64, device="cuda").bfloat16(), torch.zeros(2, 4, device="cuda")
    n = c.cache.attend_workspace_bytes(2, 4, c.table.shape[1])
    assert n > 0  # more than one cluster's, so that a workspace can be too small
    ws = torch.empty(n + 64, dtype=torch.uint8, device="cuda")
    ok = dict(q=q, table=c.table, lens=c.lens, out=torch.empty_like(q), lse=lse, workspace=ws)
    es.kv_attend(c.cache, **ok)
    wide = torch.zeros(2, 4, 128, device="cuda").bfloat16()
    for kw in (dict(q=q.half()), dict(q=q[:, :3], out=q[:, :3].clone()), dict(q=q[..., :32]), dict(q=q.cpu()), dict(q=q[0]),
               dict(q=wide[..., ::2]), dict(lens=c.lens.long()), dict(lens=c.lens[:1]), dict(lens=c.lens.cpu()),
               dict(lens=torch.stack([c.lens, c.lens], 1)[:, 0]), dict(table=c.table.long()), dict(table=c.table[:1]),
               dict(table=torch.stack([c.table, c.table], 2)[..., 0]), dict(window=-1), dict(window=2 ** 31),
               dict(window=2 ** 32 + 5), dict(out=q.float()), dict(out=q[:1]), dict(out=q.cpu()),
               dict(out=q[:, :1].expand(2, 4, 64)), dict(lse=lse.half()), dict(lse=lse.cpu()), dict(lse=lse[:, :2]),
               dict(lse=lse.t().contiguous().t()), dict(workspace=ws[:-65]), dict(workspace=ws.view(torch.int8)),
               dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            es.kv_attend(c.cache, **{**ok, **kw})
    for scale in (float("nan"), float("inf")):
        with pytest.raises(es.EStreamError):
            es.kv_attend(c.cache, **ok, scale=scale)
    want = es.kv_attend(c.cache, q, c.table, c.lens, window=7)
    assert torch.equal(es.kv_attend(c.cache, q.as_subclass(Own), c.table, c.lens, window=7, out=ok["out"]), want)
    assert torch.equal(es.kv_attend(c.cache, q, c.table, c.lens, window=7, out=ok["out"]), want)  # no workspace given

    k, n = torch.zeros(2, 2, 64, device="cuda").bfloat16(), torch.zeros(2, dtype=torch.int32, device="cuda")
    inv = torch.ones(8, device="cuda")
    good = dict(k=k, v=k, positions=n, table=c.table, rows=n, q=q, inv_freq=inv, q_out=torch.empty_like(q))
    es.kv_append(c.cache, **good)
    for kw in (dict(k=k.half()), dict(k=k[:1]), dict(k=k[:, :1]), dict(k=k.cpu()), dict(v=k.half()), dict(v=k[:, :1]), dict(v=k.cpu()),
               dict(positions=n.long()), dict(positions=n[:1]), dict(positions=n.cpu()), dict(rows=n[:1]), dict(rows=None, table=c.table[:1]),
               dict(q=None), dict(q=q.half()), dict(q=q[:1]), dict(q_out=q.float()), dict(q_out=q[:, :2]),
               dict(q_out=q[:1].expand(2, 4, 64)), dict(inv_freq=inv.double()), dict(inv_freq=inv.cpu()),
               dict(inv_freq=torch.ones(33, device="cuda")), dict(inv_freq=torch.ones(16, device="cuda")[::2])):
        with pytest.raises(ValueError):
            es.kv_append(c.cache, **{**good, **kw})

    logits, u = torch.randn(2, 100, device="cuda"), torch.rand(2, device="cuda")
    fine = dict(logits=logits, u=u, out=torch.empty(2, dtype=torch.int32, device="cuda"), prob=torch.empty(2, device="cuda"))
    es.sample_tokens(**fine)
    for kw in (dict(logits=logits.double()), dict(logits=logits.t()[:2]), dict(logits=logits[0]), dict(logits=logits.cpu()),
               dict(logits=logits[:, :0]), dict(u=u.double()), dict(u=u[:1]), dict(u=u.cpu()), dict(u=0.5), dict(out=fine["out"].long()),
               dict(out=fine["out"][:1]), dict(out=fine["out"].cpu()), dict(prob=u.double()), dict(prob=u.cpu()), dict(top_k=u),
               dict(top_k=2 ** 31), dict(top_k=2 ** 32 + 5), dict(top_p=u.double()), dict(temperature=u[:1]), dict(min_p=u.cpu())):
        with pytest.raises(ValueError):
            es.sample_tokens(**{**fine, **kw})
