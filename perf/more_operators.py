"""Cases that measure what a generation step needs next to the MoE layer: appending keys and values to a paged cache
with the position rotation on the way, attention of new tokens over such a cache, and sampling the next token.

``listed()`` names the cases, ``draw()`` gives more of the same ranges; ``prepare`` makes a case's inputs on the GPU
from a seed, ``run`` is one pass (elementary torch operations, or the library's operators where ``own`` is set),
``work`` the bytes and operations that the pass cannot do without, and ``exact`` its result in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
HALF = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}


def _attend(name, B, L, Hq, Hkv, D, page, x="bf16", kv=None, ragged=False, empty=0, window=0, by_head=False, lse=False):
    return dict(name=name, op="attend", B=B, L=L, Hq=Hq, Hkv=Hkv, D=D, page=page, x=x, kv=kv or x, ragged=ragged,
                empty=empty, window=window, by_head=by_head, lse=lse)


def _append(name, T, Hq, Hkv, D, page, x="bf16", kv=None, prompts=0, rot=None, interleaved=False, by_head=False, far=4096):
    return dict(name=name, op="append", T=T, Hq=Hq, Hkv=Hkv, D=D, page=page, x=x, kv=kv or x, prompts=prompts,
                rot=D if rot is None else rot, interleaved=interleaved, by_head=by_head, far=far)


def _sample(name, B, V, x="f32", temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, mixed=False, masked=0.0):
    return dict(name=name, op="sample", B=B, V=V, x=x, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p,
                mixed=mixed, masked=masked)


def listed():
    return [
        # one user early in a conversation: launch and synchronisation latency alone
        _attend("attend 1 x 500", 1, 500, 16, 16, 128, 16),
        # one user with a long document, four query heads to a key head: the work has to be split over the length
        _attend("attend 1 x 131072", 1, 131072, 32, 8, 128, 64, lse=True),
        # a full generation batch of conversations of all lengths, a row of padding among them
        _attend("attend 32 ragged", 32, 8192, 32, 8, 128, 16, x="f16", ragged=True, empty=1),
        # a large batch over an 8-bit cache, eight query heads to a key head, pages stored head by head
        _attend("attend 64 e4m3", 64, 16384, 64, 8, 128, 32, kv="e4m3", ragged=True, by_head=True),
        # narrow odd heads, a sliding window that starts inside a page of an odd size
        _attend("attend window", 7, 6000, 21, 3, 80, 5, x="bf16", window=1023, lse=True),
        # one generated token: latency
        _append("append 1 token", 1, 32, 8, 128, 16, far=131072),
        # a generation batch into an 8-bit cache, each sequence at a place of its own, half of each head rotated
        _append("append 32 tokens e4m3", 32, 64, 8, 128, 32, kv="e4m3", rot=64, by_head=True, far=16384),
        # four prompts, as many query heads as key heads, neighbouring values rotated together
        _append("append 4096 tokens", 4096, 16, 16, 128, 16, prompts=4, interleaved=True, far=1024),
        # one user, the default choices of a chat: temperature, top-k and top-p
        _sample("sample 1 row", 1, 50304, temperature=0.8, top_k=50, top_p=0.95),
        # a generation batch of users with choices of their own, among them greedy ones, over bf16 logits with ties
        _sample("sample 32 rows mixed", 32, 102400, x="bf16", mixed=True),
        # every row from the whole nucleus, most of the vocabulary forbidden by a grammar
        _sample("sample 64 rows top-p", 64, 32000, top_p=0.9, masked=0.7),
        # a large batch over a large vocabulary, min-p alone
        _sample("sample 256 rows min-p", 256, 151936, temperature=1.3, min_p=0.02),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "append", "sample"])
    if op == "sample":
        V = _log(rng, 1000, 200000)
        mixed = rng.random() < 0.3
        return dict(op=op, B=_log(rng, 1, max(1, min(256, 24_000_000 // V))), V=V, x=rng.choice(["f32", "f32", "bf16", "f16"]),
                    temperature=rng.choice([1.0, round(rng.uniform(0.3, 2.0), 3)]),
                    top_k=rng.choice([0, 0, _log(rng, 1, V), _log(rng, 1, 200)]),
                    top_p=rng.choice([1.0, round(rng.uniform(0.05, 1.0), 3)]),
                    min_p=rng.choice([0.0, 0.0, round(rng.uniform(0.001, 0.3), 4)]), mixed=mixed,
                    masked=rng.choice([0.0, 0.0, round(rng.uniform(0.1, 0.99), 3)]))
    Hkv, D = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128, 128, 16 * rng.randint(1, 16)])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16])
    x = rng.choice(["bf16", "bf16", "f16"])
    both = dict(op=op, Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([1, 16, 16, 64, _log(rng, 2, 256)]), x=x,
                kv=rng.choice([x, x, "e4m3"]), by_head=rng.random() < 0.5)
    if op == "attend":
        B, most = _log(rng, 1, 64), 100_000_000 // (Hkv * D)
        L = _log(rng, 1, max(1, min(65536, most // B)))
        return dict(both, B=B, L=L, ragged=rng.random() < 0.6, empty=rng.choice([0, 0, B // 3]),
                    window=rng.choice([0, 0, 0, _log(rng, 1, L)]), lse=rng.random() < 0.5)
    T = _log(rng, 1, min(8192, 20_000_000 // ((Hq + Hkv) * D)))
    far = _log(rng, 64, max(64, min(131072, 8_000_000 // T * both["page"])))
    return dict(both, T=T, prompts=rng.choice([0, 1, 3]) if T >= 3 else 0, far=far, rot=rng.choice([D, D, 2 * rng.randint(0, D // 2)]),
                interleaved=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)


def _randn(g, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _lens(c):
    """The sequences' lengths before they are shuffled: all L, or spread from short to L; the first ones empty."""
    n = [c["L"]] * c["B"]
    if c["ragged"]:
        n = [max(1, math.ceil(c["L"] * ((i + 1) / c["B"]) ** 2)) for i in range(c["B"])]
    return [0] * c["empty"] + n[c["empty"]:]


def _pages(g, c, pages, std):
    """A cache's keys or values [pages, page, Hkv, D], stored token by token or head by head, and their scale."""
    scale = 2.0 ** -6 if c["kv"] == "e4m3" else 1.0
    shape = (pages, c["Hkv"], c["page"], c["D"]) if c["by_head"] else (pages, c["page"], c["Hkv"], c["D"])
    t = _randn(g, shape, std / scale, HALF["f16"] if c["kv"] == "e4m3" else HALF[c["kv"]])
    t = t.float().clamp(-448.0, 448.0).to(HALF["e4m3"]) if c["kv"] == "e4m3" else t
    return (t.transpose(1, 2) if c["by_head"] else t), scale


def _cache(g, c, pages):
    (k, ks), (v, vs) = _pages(g, c, pages, 1.0), _pages(g, c, pages, 1.0)
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}


def _prepare_attend(c, g):
    order = torch.randperm(c["B"], generator=g, device=DEV)
    lens = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)[order]
    M = -(-max(1, c["L"]) // c["page"])
    used = (lens + c["page"] - 1) // c["page"]
    pages = sum(-(-n // c["page"]) for n in _lens(c)) + 3
    # pages in the order in which an allocator that serves many users hands them out; none past a sequence's end
    first = used.cumsum(0) - used
    at = first[:, None] + torch.arange(M, device=DEV)
    has = torch.arange(M, device=DEV) < used[:, None]
    shuffled = torch.randperm(pages, generator=g, device=DEV)
    table = torch.where(has, shuffled[torch.where(has, at, 0)], -1).to(torch.int32)
    # scores that spread over a few units: some keys stand out, the many others add up
    q = _randn(g, (c["B"], c["Hq"], c["D"]), 2.5, HALF[c["x"]])
    return dict(_cache(g, c, pages), q=q, table=table, lens=lens, out=torch.empty_like(q),
                lse=torch.empty(c["B"], c["Hq"], device=DEV) if c["lse"] else None)


def _prepare_append(c, g):
    T, far = c["T"], c["far"]
    n = c["prompts"]
    if n:  # whole prompts, one behind another
        rows = torch.arange(T, device=DEV) * n // T
        start = torch.searchsorted(rows, torch.arange(n, device=DEV))
        positions = torch.arange(T, device=DEV) - start[rows]
        B, M = n, -(-(T // n + 1) // c["page"])
    else:  # one new token of each sequence, at the end of it
        rows, B = None, T
        positions = torch.randint(0, far, (T,), generator=g, device=DEV)
        M = -(-far // c["page"])
    # the pages that this step writes, and a few of other users'; further ones are not there
    if n:
        pages = B * M + 3
        table = torch.randperm(pages, generator=g, device=DEV)[:B * M].view(B, M)
    else:
        pages = B + 3
        table = torch.full((B, M), -1, device=DEV)
        table.scatter_(1, (positions // c["page"])[:, None], torch.randperm(pages, generator=g, device=DEV)[:B, None])
    qkv = _randn(g, (T, c["Hq"] + 2 * c["Hkv"], c["D"]), 1.0, HALF[c["x"]])
    inv = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / max(1, c["rot"]))
    return dict(_cache(g, c, pages), qkv=qkv, positions=positions.to(torch.int32), table=table.to(torch.int32),
                rows=None if rows is None else rows.to(torch.int32), inv_freq=inv.float() if c["rot"] else None,
                q_out=torch.empty(T, c["Hq"], c["D"], dtype=HALF[c["x"]], device=DEV))


def _prepare_sample(c, g):
    B, V = c["B"], c["V"]
    # a bulk that is common to all rows, and a few tokens of each that stand out
    logits = _randn(g, (B, V), 2.0) + _randn(g, (1, V), 1.5)
    hot = torch.randint(0, V, (B, min(V, 20)), generator=g, device=DEV)
    logits.scatter_add_(1, hot, _randn(g, hot.shape, 2.0) + 8.0)
    if c["masked"]:
        logits = torch.where(torch.rand(B, V, generator=g, device=DEV) < c["masked"], float("-inf"), logits)
    s = dict(logits=logits.to(HALF[c["x"]]), u=torch.rand(B, generator=g, device=DEV))
    s["choice"] = {n: c[n] for n in ("temperature", "top_k", "top_p", "min_p")}
    if c["mixed"]:  # a value for each row
        r = torch.rand(4, B, generator=g, device=DEV)
        t = torch.where(r[0] < 0.2, 0.0, 0.5 + r[0])
        s["choice"] = dict(temperature=t, top_k=torch.where(r[1] < 0.4, 0.0, torch.exp(r[1] * 7.0)).to(torch.int32),
                           top_p=torch.where(r[2] < 0.4, 1.0, r[2]), min_p=torch.where(r[3] < 0.6, 0.0, 0.1 * r[3]))
    s["ids"] = torch.empty(B, dtype=torch.int32, device=DEV)
    s["prob"] = torch.empty(B, device=DEV)
    return s


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"attend": _prepare_attend, "append": _prepare_append, "sample": _prepare_sample}[c["op"]](c, g)
    s["case"] = c
    if own and c["op"] != "sample":
        from routed_expert_ffn_topk_gb300 import estream as es
        s["cache"] = es.PagedKV(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def _rows_of(pages, table):
    """The pages of a table's rows behind one another: [B, M * page, Hkv, D] in 32 bits; entry -1 reads page 0."""
    t = table.clamp(min=0).long()
    if pages.dtype == torch.float8_e4m3fn:
        return pages.view(torch.uint8)[t].view(torch.float8_e4m3fn).float().flatten(1, 2)
    return pages[t].float().flatten(1, 2)


def _attend_plain(s):
    c = s["case"]
    B, Hq, D = s["q"].shape
    k, v = _rows_of(s["k"], s["table"]) * s["k_scale"], _rows_of(s["v"], s["table"]) * s["v_scale"]
    at = torch.arange(k.shape[1], device=k.device)
    seen = at < s["lens"][:, None]
    if c["window"]:
        seen = seen & (at >= s["lens"][:, None] - c["window"])
    q = s["q"].float().view(B, c["Hkv"], -1, D)
    score = (q @ k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    score = score.masked_fill(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = v.masked_fill(~seen[:, :, None, None], 0.0)
    o = (p @ v.transpose(1, 2)) / torch.where(total > 0, total, torch.ones_like(total))
    out = {"out": o.view(B, Hq, D).to(s["q"].dtype)}
    if c["lse"]:
        out["lse"] = (top + torch.log(total)).view(B, Hq)
    return out


def _attend_own(s):
    from routed_expert_ffn_topk_gb300 import estream as es
    c = s["case"]
    es.kv_attend(s["cache"], s["q"], s["table"], s["lens"], window=c["window"], out=s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]} if c["lse"] else {"out": s["out"]}


def _split(c, qkv):
    return qkv[:, :c["Hq"]], qkv[:, c["Hq"]:c["Hq"] + c["Hkv"]], qkv[:, c["Hq"] + c["Hkv"]:]


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    if not rot:
        return x
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    cos, sin = cos[:, None], sin[:, None]
    lo, hi = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([lo, hi], -1).flatten(-2) if interleaved else torch.cat([lo, hi], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _stored(x, scale, dtype):
    if dtype == torch.float8_e4m3fn:
        return (x * (1.0 / scale)).clamp(-448.0, 448.0).to(dtype)
    return x.to(dtype)


def _put(pages, page, off, x):
    """Rows of x into their places; bytes where the type is of 8 bits."""
    if pages.dtype == torch.float8_e4m3fn:
        pages.view(torch.uint8)[page, off] = x.view(torch.uint8)
    else:
        pages[page, off] = x


def _append_plain(s):
    c = s["case"]
    q, k, v = _split(c, s["qkv"])
    pos = s["positions"].long()
    cos = sin = None
    if c["rot"]:  # angles of far positions in 64 bits
        angle = pos[:, None].double() * s["inv_freq"].double()
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    rows = torch.arange(c["T"], device=pos.device) if s["rows"] is None else s["rows"].long()
    page, off = s["table"][rows, pos // c["page"]].long(), pos % c["page"]
    _put(s["k"], page, off, _stored(_rotate(k, cos, sin, c["rot"], c["interleaved"]), s["k_scale"], s["k"].dtype))
    _put(s["v"], page, off, _stored(v.float(), s["v_scale"], s["v"].dtype))
    return {"k": s["k"], "v": s["v"], "q": _rotate(q, cos, sin, c["rot"], c["interleaved"]).to(q.dtype)}


def _append_own(s):
    from routed_expert_ffn_topk_gb300 import estream as es
    c = s["case"]
    q, k, v = _split(c, s["qkv"])
    es.kv_append(s["cache"], k, v, s["positions"], s["table"], rows=s["rows"], q=q, q_out=s["q_out"],
                 inv_freq=s["inv_freq"], interleaved=c["interleaved"])
    return {"k": s["k"], "v": s["v"], "q": s["q_out"]}


def _column(x, like, dtype):
    """A choice of all rows or of each, as [B, 1]; a number is one of 32 bits, as the call takes it."""
    t = x if torch.is_tensor(x) else torch.full((like.shape[0],), x, dtype=torch.float32, device=like.device)
    return t.to(dtype)[:, None]


def _sample_plain(s):
    # in 64 bits: a token's place among 10^5 others is next to a border
    l = s["logits"].double()
    B, V = l.shape
    ch = s["choice"]
    t, p, low = (_column(ch[n], l, torch.float64) for n in ("temperature", "top_p", "min_p"))
    kk = _column(ch["top_k"], l, torch.int64)
    greedy = ~(t > 0)
    top = l.amax(1, keepdim=True)
    ranked, order = torch.sort(l, dim=1, descending=True, stable=True)
    w = torch.exp((ranked - top) / torch.where(greedy, torch.ones_like(t), t))
    rank = torch.arange(V, device=l.device)[None]
    keep = (rank < kk) | (kk <= 0)
    w = torch.where(keep, w, torch.zeros_like(w))
    before = w.cumsum(1) - w
    keep = keep & ((before < p * w.sum(1, keepdim=True)) | (p >= 1.0)) & (w >= low * w[:, :1]) | (rank == 0)
    w = torch.where(keep, w, torch.zeros_like(w))
    w = torch.zeros_like(w).scatter_(1, order, w)  # back in the vocabulary's order
    upto = w.cumsum(1)
    total = upto[:, -1:]
    hit = (upto > s["u"].double()[:, None] * total) & (w > 0)
    ids = hit.to(torch.uint8).argmax(1, keepdim=True)  # the first of the largest
    prob = torch.where(greedy, torch.ones_like(total), w.gather(1, ids) / total)
    ids = torch.where(greedy, (l == top).to(torch.uint8).argmax(1, keepdim=True), ids)
    return {"ids": ids[:, 0].to(torch.int32), "prob": prob[:, 0].float()}


def _sample_own(s):
    from routed_expert_ffn_topk_gb300 import estream as es
    es.sample_tokens(s["logits"], s["u"], **s["choice"], out=s["ids"], prob=s["prob"])
    return {"ids": s["ids"], "prob": s["prob"]}


def run(state):
    return {("attend", False): _attend_plain, ("attend", True): _attend_own, ("append", False): _append_plain,
            ("append", True): _append_own, ("sample", False): _sample_plain,
            ("sample", True): _sample_own}[state["case"]["op"], bool(own)](state)


def work(case):
    c = case
    if c["op"] == "attend":
        n = sum(min(x, c["window"]) if c["window"] else x for x in _lens(c))
        b = 2 * n * c["Hkv"] * c["D"] * SIZE[c["kv"]] + 2 * c["B"] * c["Hq"] * c["D"] * SIZE[c["x"]]
        b += 4 * c["B"] + 4 * (n // c["page"]) + (4 * c["B"] * c["Hq"] if c["lse"] else 0)
        return {"bytes": b, "flops": 4.0 * n * c["Hq"] * c["D"]}
    if c["op"] == "append":
        b = c["T"] * c["D"] * ((2 * c["Hq"] + 2 * c["Hkv"]) * SIZE[c["x"]] + 2 * c["Hkv"] * SIZE[c["kv"]])
        return {"bytes": b + 8 * c["T"] + 2 * c["rot"], "flops": 3.0 * c["T"] * c["rot"] * (c["Hq"] + c["Hkv"])}
    return {"bytes": c["B"] * (c["V"] * SIZE[c["x"]] + 12), "flops": 4.0 * c["B"] * c["V"]}


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def _at(pages, page, off, h):
    """Rows [n, D] of one head in 64 bits."""
    if pages.dtype == torch.float8_e4m3fn:
        return pages.view(torch.uint8)[page, off, h].view(torch.float8_e4m3fn).double()
    return pages[page, off, h].double()


def _exact_attend(c, s):
    B, Hq, D, G = c["B"], c["Hq"], c["D"], c["Hq"] // c["Hkv"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq), float("-inf"), dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        at = torch.arange(max(0, n - c["window"]) if c["window"] else 0, n, device=DEV)
        if not len(at):
            continue
        page, off = s["table"][b].long()[at // c["page"]], at % c["page"]
        for h in range(c["Hkv"]):
            mine = slice(h * G, (h + 1) * G)
            z = s["q"][b, mine].double() @ _at(s["k"], page, off, h).t() * (s["k_scale"] / math.sqrt(D))
            lse[b, mine] = torch.logsumexp(z, 1)
            out[b, mine] = torch.softmax(z, 1) @ _at(s["v"], page, off, h) * s["v_scale"]
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def _to_e4m3(x):
    """To 4 significant bits, or to multiples of 2^-9 below 2^-6, ties to even, at most 448."""
    ulp = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3.0)
    return (torch.round(x / ulp) * ulp).clamp(-448.0, 448.0)


def _exact_append(c, s):
    T, Hq, Hkv, rot = c["T"], c["Hq"], c["Hkv"], c["rot"]
    x = s["qkv"].double()
    if rot:
        angle = torch.einsum("t,i->ti", s["positions"].double(), s["inv_freq"].double())
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        for lo, hi in ((0, Hq), (Hq, Hq + Hkv)):
            part = x[:, lo:hi, :rot]
            if c["interleaved"]:
                z = torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous()) * turn
                x[:, lo:hi, :rot] = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(part[..., :rot // 2], part[..., rot // 2:]) * turn
                x[:, lo:hi, :rot] = torch.cat([z.real, z.imag], -1)
    out = {"q": x[:, :Hq]}
    for name, part in (("k", x[:, Hq:Hq + Hkv]), ("v", x[:, Hq + Hkv:])):
        part = _to_e4m3(part / s[name + "_scale"]) if c["kv"] == "e4m3" else part
        pages = s[name].float().double()
        for t, p in enumerate(s["positions"].tolist()):
            row = t if s["rows"] is None else int(s["rows"][t])
            pages[int(s["table"][row, p // c["page"]]), p % c["page"]] = part[t]
        out[name] = pages
    return out


def _exact_sample(c, s):
    ids, probs = [], []
    for b in range(c["B"]):
        one = {n: (x[b] if torch.is_tensor(x) else torch.tensor(x, dtype=torch.float32)).item() for n, x in s["choice"].items()}
        l = s["logits"][b].double()
        best = int((l == l.max()).nonzero()[0])
        if not one["temperature"] > 0:
            ids.append(best)
            probs.append(1.0)
            continue
        # likeliest first, then lower index first
        order = torch.argsort(-l, stable=True)
        if one["top_k"] > 0:
            order = order[:int(one["top_k"])]
        w = torch.exp((l[order] - l[best]) / one["temperature"])
        n = len(order)
        if one["top_p"] < 1:
            n = max(1, int((torch.cat([w.new_zeros(1), w.cumsum(0)[:-1]]) < one["top_p"] * w.sum()).sum()))
        n = max(1, min(n, int((w >= one["min_p"]).sum())))
        kept, back = torch.sort(order[:n])
        share = w[:n][back] / w[:n].sum()
        at = min(int((share.cumsum(0) <= s["u"][b].double()).sum()), n - 1)
        ids.append(int(kept[at]))
        probs.append(float(share[at]))
    return {"ids": torch.tensor(ids, dtype=torch.int32, device=DEV),
            "prob": torch.tensor(probs, dtype=torch.float64, device=DEV)}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"attend": _exact_attend, "append": _exact_append, "sample": _exact_sample}[case["op"]](case, s)
