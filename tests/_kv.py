"""Paged caches and the formulas of the cache's calls in 64 bits, for their tests."""
import math

import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def pages(n, page, heads, dim, kind, by_head=False, fill=float("nan"), device="cuda"):
    """An empty cache's keys or values [n, page, heads, dim], every element `fill`."""
    shape = (n, heads, page, dim) if by_head else (n, page, heads, dim)
    t = torch.full(shape, fill, device=device).to(DT[kind])
    return t.transpose(1, 2) if by_head else t


def put(t, page, slot, x):
    """Rows x [n, heads, dim] into a cache's places."""
    if t.dtype == torch.float8_e4m3fn:
        t.view(torch.uint8)[page, slot] = x.to(t.dtype).view(torch.uint8)
    else:
        t[page, slot] = x.to(t.dtype)


def get(t, page, slot):
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).double()
    return t[page, slot].double()


class Case:
    """Sequences of the given lengths in a cache that holds NaN wherever nothing was
    put, their pages in random order, -1 in the table past a sequence's end."""

    def __init__(self, lens, heads, dim, page, kind, by_head=False, M=None, seed=0, scales=(1.0, 1.0), window=0,
                 first_page=0):
        g = torch.Generator().manual_seed(seed)
        self.lens_list, self.window = lens, window
        B, L = len(lens), max(max(lens), 1)
        M = -(-L // page) if M is None else M
        used = [-(-n // page) for n in lens]
        n = sum(used) + 2 + first_page
        order = (torch.randperm(n - first_page, generator=g) + first_page).tolist()
        table = torch.full((B, M), -1, dtype=torch.int32)
        self.k, self.v = pages(n, page, heads, dim, kind, by_head), pages(n, page, heads, dim, kind, by_head)
        self.place = []
        for b, count in enumerate(lens):
            mine = [order.pop() for _ in range(used[b])]
            table[b, :used[b]] = torch.tensor(mine, dtype=torch.int32)
            at = torch.arange(max(0, count - window) if window else 0, count)
            p, s = torch.tensor(mine, dtype=torch.long)[at // page].cuda(), (at % page).cuda()
            for t, scale in ((self.k, scales[0]), (self.v, scales[1])):
                put(t, p, s, torch.randn(len(at), heads, dim, generator=g).cuda() / scale)
            self.place.append((p, s))
        self.table, self.lens = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        self.scales = scales
        from routed_expert_ffn_topk_gb300 import estream as es
        self.cache = es.PagedKV(self.k, self.v, *scales)

    def want(self, q, scale):
        """out, lse in 64 bits, and the bound of each value's error (see attend_bounds)."""
        B, Hq, D = q.shape
        heads = self.k.shape[2]
        G = Hq // heads
        out, lse = torch.zeros(B, Hq, D, dtype=torch.float64), torch.full((B, Hq), -math.inf, dtype=torch.float64)
        tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
        kind = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float8_e4m3fn: "e4m3"}[self.k.dtype]
        for b, (p, s) in enumerate(self.place):
            if not len(p):
                continue
            k, v = get(self.k, p, s) * self.scales[0], get(self.v, p, s) * self.scales[1]
            for h in range(Hq):
                kk, vv, qq = k[:, h // G], v[:, h // G], q[b, h].double()
                z = kk @ qq * scale
                w = torch.softmax(z, 0)
                out[b, h], lse[b, h] = (w @ vv).cpu(), float(torch.logsumexp(z, 0))
                size = float((kk.abs() @ qq.abs()).max()) * abs(scale)
                tol[b, h], ltol[b, h] = attend_bounds(out[b, h], (w @ vv.abs()).cpu(), float(vv.abs().max()), lse[b, h], len(p), D,
                                                      size, kind, q.dtype)
        return out, lse, tol, ltol


def attend_bounds(out, mean, most, lse, n, D, size, kind, dtype):
    """Bounds of attention's errors. A score is a sum of D exact products in fp32, each addition off
    by at most 2^-23 (matrix instructions truncate) of the sum of magnitudes: D 2^-23 size, and 2^-22
    of itself for the two roundings to base 2. A weight is off by that, 2^-22 (exponential), and its
    rounding: 2^-16 for bf16's two terms, else 2^-11 or half of 2^-38 of the largest. It enters the
    value's numerator and denominator. Sums over n positions in chains of n / 16 + 64 additions.
    The result is rounded once; fp16's smallest step is 2^-24."""
    dz = (D + 2) * 2.0 ** -23 * size + 2.0 ** -22 * size
    dw = dz + 2.0 ** -22
    chain = (n / 16 + 64) * 2.0 ** -23
    round_w = 2.0 ** -16 if kind == "bf16" else 2.0 ** -11
    tiny = 0.0 if kind == "bf16" else n * 2.0 ** -39 * most
    u = torch.finfo(dtype).eps / 2
    tol = (mean * (2 * dw + round_w + 2 * chain) + tiny + 1e-30) * (1 + u) + u * out.abs() + 2.0 ** -25
    return tol, dw + chain + 2.0 ** -22 * abs(lse) + 2.0 ** -21


def rotate64(x, pos, inv_freq, interleaved):
    """Rows x [T, heads, dim] in 64 bits turned by pos * inv_freq; and |a| + |b| of each value's pair."""
    y, size, rot = x.clone(), torch.zeros_like(x), 2 * len(inv_freq)
    t = (pos.double()[:, None] * inv_freq.double())[:, None]
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., a] = x[..., a] * t.cos() - x[..., b] * t.sin()
    y[..., b] = x[..., b] * t.cos() + x[..., a] * t.sin()
    size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size
