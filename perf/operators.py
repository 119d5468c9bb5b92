"""Cases that measure the few-token MoE layer and the microscaled 4-bit operators.

``listed()`` names the cases, ``draw()`` gives more of the same ranges; ``prepare`` makes a case's inputs on the GPU
from a seed, ``run`` is one pass (elementary torch operations, or the library's operators where ``own`` is set),
``work`` the bytes and operations that the pass cannot do without, and ``exact`` its result in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
HALF = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = {"e4m3": 16, "e8m0": 32}  # values that share a scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _layer(name, w, T, H, E, k, F, renorm=False, n_shared=0, F_shared=0, router=False, residual=True):
    return dict(name=name, op="decode", w=w, T=T, H=H, E=E, k=k, F=F, renorm=renorm, n_shared=n_shared,
                F_shared=F_shared, router=router, residual=residual)


def _quant(name, R, K, x, fmt, src=0, swiglu=False):
    return dict(name=name, op="quantize", R=R, K=K, x=x, fmt=fmt, src=src, swiglu=swiglu)


def _prod(name, R, N, K, fmt, P=1, out="bf16"):
    return dict(name=name, op="product", R=R, N=N, K=K, fmt=fmt, P=P, out=out)


def listed():
    return [
        # the tiny fp32 layer, one generated token: launch and synchronisation latency alone
        _layer("layer tiny f32 1 token", "f32", 1, 256, 8, 2, 512),
        # one generated token through the OLMoE-shaped layer, router included: the step of a single user
        _layer("layer olmoe 1 token", "bf16", 1, 2048, 64, 8, 1024, router=True),
        # four sequences, renormalised weights and two shared experts (DeepSeek-V2-Lite shape)
        _layer("layer deepseek 4 tokens", "bf16", 4, 2048, 64, 6, 1408, renorm=True, n_shared=2, F_shared=1408),
        # two sequences through the largest experts (Mixtral shape) kept as 4-bit integers
        _layer("layer mixtral q4 2 tokens", "q4", 2, 4096, 8, 2, 14336, renorm=True),
        # a full generation batch: nearly every expert is read, several tokens each
        _layer("layer olmoe 32 tokens", "bf16", 32, 2048, 64, 8, 1024),
        # one token's activations ahead of a product
        _quant("quantize 1 row", 1, 2048, "bf16", "e4m3"),
        # a prompt's rows gathered by the route map (1024 tokens, 8 routes each), ahead of the gate/up product
        _quant("quantize gathered rows", 8192, 2048, "bf16", "e4m3", src=1024),
        # SwiGLU of the gate/up product's rows, ahead of the down product
        _quant("quantize swiglu rows", 8192, 14336, "bf16", "e8m0", swiglu=True),
        # a dense projection of one token
        _prod("product 1 row", 1, 14336, 4096, "e8m0"),
        # the same projection of a ragged batch, fp32 out
        _prod("product 333 rows", 333, 5632, 2048, "e4m3", out="f32"),
        # the gate and up products of a prompt over 64 experts, records grouped by the route map
        _prod("product grouped", 8192, 2048, 2048, "e4m3", P=64),
        # the largest dense product of a prompt
        _prod("product 4096 rows", 4096, 14336, 4096, "e4m3"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "quantize", "product"])
    if op == "decode":
        w = rng.choice(["bf16", "bf16", "q4", "f32"])
        H = 256 * _log(rng, 1, 16 if w != "f32" else 4)
        F = 128 * _log(rng, 1, 24 if w != "f32" else 8)
        E = _log(rng, 2, 64)
        while E * H * F > 140_000_000:
            E = max(2, E // 2)
        T = _log(rng, 1, 32)
        shared = rng.choice([0, 0, 1, 2])
        return dict(op=op, w=w, T=T, H=H, E=E, k=rng.randint(1, min(8, E)), F=F, renorm=rng.random() < 0.5,
                    n_shared=shared, F_shared=128 * rng.randint(1, 8) if shared else 0,
                    router=w != "f32" and T <= 4 and rng.random() < 0.5, residual=rng.random() < 0.8)
    fmt = rng.choice(["e4m3", "e8m0"])
    if op == "quantize":
        swiglu = rng.random() < 0.4
        K = _log(rng, 16, 4096) if swiglu else _log(rng, 1, 16384)
        R = _log(rng, 1, max(1, min(16384, 60_000_000 // K)))
        return dict(op=op, R=R, K=K, x=rng.choice(["bf16", "bf16", "f16", "f32"]), fmt=fmt,
                    src=rng.choice([0, max(1, R // rng.randint(1, 8))]), swiglu=swiglu)
    P = rng.choice([1, 1, 8, 60])
    N, K = _log(rng, 64, 8192 if P == 1 else 2816), _log(rng, 64, 8192 if P == 1 else 2048)
    return dict(op=op, R=_log(rng, 1, 4096), N=N, K=K, fmt=fmt, P=P, out=rng.choice(["bf16", "bf16", "f32"]))


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)


def _randn(g, shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _to_5_bits(x):
    """fp32 rounded to 5 significant bits, ties to even."""
    u = x.view(torch.int32)
    low = u & 0x7FFFF
    u = u - low
    up = (low > 0x40000) | ((low == 0x40000) & ((u >> 19) & 1 == 1))
    return (u + up.to(torch.int32) * (1 << 19)).view(torch.float32)


def _q4(w):
    """4-bit integer blocks of 32 along the last dimension: codes [..., n/32, 32] and scales [..., n/32, 1]."""
    b = w.float().unflatten(-1, (-1, 32))
    m = b.gather(-1, b.abs().argmax(-1, keepdim=True))
    d = _to_5_bits(m / -8.0)
    q = torch.where(d == 0, torch.full_like(b, 8.0), (torch.round(b / d) + 8).clamp(0, 15))
    return q, d


def _experts(g, n, H, F, w):
    """Gate and up [n, F, H], down [n, H, F] of a layer, and the 4-bit form of each where the layer has it."""
    dt = torch.float32 if w == "f32" else torch.bfloat16
    out, packed = [], []
    for shape in ((n, F, H), (n, F, H), (n, H, F)):
        t = torch.empty(shape, dtype=dt, device=DEV)
        t.normal_(0.0, 0.02, generator=g)
        if w == "q4":
            qd = [_q4(t[e]) for e in range(n)]
            for e, (q, d) in enumerate(qd):
                t[e] = ((q - 8) * d).flatten(-2).to(dt)
            packed.append([(q.to(torch.uint8), d) for q, d in qd])
        out.append(t)
    return out, packed


def _tiles(w, rows):
    """One expert's [N, K] plane as [N/rows][K/64][rows][64]."""
    N, K = w.shape
    return w.view(N // rows, rows, K // 64, 64).permute(0, 2, 1, 3).contiguous()


def _q4_tiles(q, d, rows, bits):
    """One expert's 4-bit plane as tile-major boxes: two column blocks of codes, then the rows' scales."""
    N, nb = q.shape[0], q.shape[1]
    c = q.view(N // rows, rows, nb // 2, 2, 4, 4, 2).to(torch.int64)  # row tile, row, k-box, block, word, i, parity
    i = torch.arange(4, device=DEV)
    word = (c[..., 0] << (4 * i)).sum(-1) + (c[..., 1] << (16 + 4 * i)).sum(-1)
    word = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
    codes = word.permute(0, 2, 3, 1, 4).contiguous().view(N // rows, nb // 2, rows * 8).view(torch.uint8)
    s = d.view(N // rows, rows, nb // 2, 2).permute(0, 2, 1, 3).contiguous().to(bits)
    return torch.cat([codes, s.view(N // rows, nb // 2, rows * 2).view(torch.uint8)], dim=-1)


def _planes(ws, packed, w):
    """The three planes of n experts as the library keeps them, and the down scales."""
    n = ws[0].shape[0]
    if w == "f32":
        return [t.view(torch.uint8).reshape(-1) for t in ws], torch.ones(n)
    planes, scales = [], torch.ones(n)
    for j, t in enumerate(ws):
        rows = 256 if j == 2 else 128
        parts = []
        for e in range(n):
            s = 0
            if j == 2:
                top = float(t[e].abs().max())
                s = 15 - math.frexp(top)[1] if top > 0 else 0
                scales[e] = math.ldexp(1.0, -s)
            if w == "q4":
                q, d = packed[j][e]
                parts.append(_q4_tiles(q, d * 2.0 ** s, rows, torch.float16 if j == 2 else torch.bfloat16).reshape(-1))
            else:
                u = (t[e].float() * 2.0 ** s).half() if j == 2 else t[e]
                parts.append(_tiles(u, rows).view(torch.uint8).reshape(-1))
        planes.append(torch.cat(parts))
    return planes, scales


class _Bound:
    """A layer bound for generation: its resident arena, host pool and context, as a serving program keeps them."""

    def __init__(self, c, ws, packed, shared, shared_packed):
        from routed_expert_ffn_topk_gb300 import estream as es
        self.es = es
        wd = {"f32": es.F32, "bf16": es.BF16, "q4": es.Q4}[c["w"]]
        E, H, F = c["E"], c["H"], c["F"]
        planes, scales = _planes(ws, packed, c["w"])
        self.pool = torch.zeros(es.pool_bytes(E, H, F, wd), dtype=torch.uint8, pin_memory=True)
        at = 0
        for p in planes + [scales.view(torch.uint8)]:
            self.pool[at:at + p.numel()].copy_(p)
            at += p.numel()
        self.shared = None
        if c["n_shared"]:
            planes, scales = _planes(shared, shared_packed, c["w"])
            buf = torch.zeros(es.shared_bytes(c["n_shared"], H, c["F_shared"], wd), dtype=torch.uint8, device=DEV)
            at = 0
            for p in planes + [scales.view(torch.uint8).to(DEV)]:
                buf[at:at + p.numel()].copy_(p)
                at += p.numel()
            self.shared = [buf]
        self.arena = torch.empty(es.arena_bytes(E, H, F, E, 1, wd), dtype=torch.uint8, device=DEV)
        desc, self.keep = es.make_desc(1, E, H, F, E, 1, wd, self.arena, [self.pool], n_shared=c["n_shared"],
                                       F_shared=c["F_shared"], shared=self.shared, T_max=32, k_max=c["k"])
        torch.cuda.synchronize()
        self.ctx = es.bind_arena(desc)
        es.arena_preload(self.ctx, 0)

    def __del__(self):
        if getattr(self, "ctx", None):
            torch.cuda.synchronize()
            self.es.unbind(self.ctx)
            self.ctx = None


def _scale_bytes(g, shape, fmt):
    """Block scales of data of about unit size, as bytes: E4M3 between 0.2 and 0.7, or 2^-4 .. 2^-1."""
    if fmt == "e8m0":
        return torch.randint(123, 127, shape, generator=g, device=DEV, dtype=torch.uint8)
    return torch.randint(0x25, 0x33, shape, generator=g, device=DEV, dtype=torch.uint8)


def _padded(K):
    return -(-K // 32) * 32


def _codes(g, shape, K):
    """Random codes, two to a byte, low half first; zeros past K."""
    c = torch.randint(0, 256, (*shape, _padded(K) // 2), generator=g, device=DEV, dtype=torch.uint8)
    c[..., (K + 1) // 2:] = 0
    if K % 2:
        c[..., K // 2] &= 0x0F
    return c


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "decode":
        T, H, E, k = c["T"], c["H"], c["E"], c["k"]
        ws, packed = _experts(g, E, H, c["F"], c["w"])
        shared, sp = _experts(g, c["n_shared"], H, c["F_shared"], c["w"]) if c["n_shared"] else (None, None)
        dt = torch.float32 if c["w"] == "f32" else torch.bfloat16
        s["X"] = _randn(g, (T, H), 1.0, dt)
        s["logits"] = _randn(g, (T, E)) + _randn(g, (1, E), 0.5)
        s["W_r"] = _randn(g, (E, H), 1.0 / math.sqrt(H), torch.bfloat16) if c["router"] else None
        if own:
            s["bound"] = _Bound(c, ws, packed, shared, sp)
            s["Y"] = torch.empty(T, H, device=DEV)
        else:
            s["W"], s["S"] = ws, shared
    elif c["op"] == "quantize":
        n, width = c["src"] or c["R"], c["K"] * (2 if c["swiglu"] else 1)
        # a few channels are much larger than the others, as activations have them
        x = _randn(g, (n, width)) * torch.exp(_randn(g, (1, width), 0.7))
        s["x"] = x.to(HALF[c["x"]])
        s["rows"] = None
        if c["src"]:
            s["rows"] = torch.randint(0, n, (c["R"],), generator=g, device=DEV, dtype=torch.int32)
        s["scale"] = 2.0 ** -4 if c["fmt"] == "e4m3" else 1.0
    else:
        R, N, K, P, b = c["R"], c["N"], c["K"], c["P"], BLOCK[c["fmt"]]
        nb = _padded(K) // b
        xc, xs = _codes(g, (R,), K), _scale_bytes(g, (R, nb), c["fmt"])
        wc, wsc = _codes(g, (P, N), K), _scale_bytes(g, (P, N, nb), c["fmt"])
        s["scale"] = 2.0 ** -3, 2.0 ** -5
        s["offsets"] = None
        if P > 1:  # records of each slot: skewed, some slots empty
            p = torch.softmax(_randn(g, (P,), 0.5), 0)
            n = torch.bincount(torch.multinomial(p, R, True, generator=g), minlength=P)
            s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
        if own:
            from routed_expert_ffn_topk_gb300 import estream as es
            fmt = es.FP4_E4M3X16 if c["fmt"] == "e4m3" else es.FP4_E8M0X32
            s["x"] = es.Mx4(xc, xs, K, fmt, s["scale"][0])
            s["w"] = es.mx4_weights(wc, wsc, K, fmt, s["scale"][1])
        else:
            s["x"], s["w"] = (xc, xs), (wc, wsc)
            s["cap"] = int((s["offsets"][1:] - s["offsets"][:-1]).max()) if P > 1 else R
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def _silu(x):
    return x / (1.0 + torch.exp(-x))


def _layer_plain(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = s["X"].float()
    lg = x @ s["W_r"].float().t() if c["router"] else s["logits"]
    p = torch.exp(lg - lg.max(1, keepdim=True).values)
    p = p / p.sum(1, keepdim=True)
    ids = torch.sort(lg, dim=1, descending=True, stable=True).indices[:, :k]
    a = p.gather(1, ids)
    if c["renorm"]:
        a = a / a.sum(1, keepdim=True)
    Wg, Wu, Wd = s["W"]
    if T * k <= E:  # few routes: each one's weights
        h = _silu(Wg[ids].float() @ x[:, None, :, None]) * (Wu[ids].float() @ x[:, None, :, None])
        y = ((Wd[ids].float() @ h)[..., 0] * a[..., None]).sum(1)
    else:  # every expert over every token, weight zero where it was not chosen
        F = c["F"]
        full = torch.zeros(T, E, device=x.device).scatter_(1, ids, a)
        h = _silu(x @ Wg.view(E * F, -1).float().t()) * (x @ Wu.view(E * F, -1).float().t())
        h = (h.view(T, E, F) * full[..., None]).view(T, E * F)
        y = h @ Wd.float().transpose(1, 2).reshape(E * F, -1)
    if c["n_shared"]:
        Sg, Su, Sd = (t.float() for t in s["S"])
        n, F = Sg.shape[:2]
        h = _silu(x @ Sg.view(n * F, -1).t()) * (x @ Su.view(n * F, -1).t())
        y = y + h @ Sd.transpose(1, 2).reshape(n * F, -1)
    y = x + y if c["residual"] else y
    return {"y": y, "logits": lg} if c["router"] else {"y": y}


def _layer_own(s):
    from routed_expert_ffn_topk_gb300 import estream as es
    c, Y = s["case"], s["Y"]
    A = s["X"] if c["residual"] else None
    if A is None:
        Y.zero_()
    if not c["router"]:
        es.moe_layer_decode(s["bound"].ctx, 0, s["X"], s["logits"], c["k"], c["renorm"], Y, A=A)
        return {"y": Y}
    lg = torch.empty(c["T"], c["E"], device=DEV)
    es.moe_layer_decode_from_x(s["bound"].ctx, 0, s["X"], s["W_r"], c["k"], c["renorm"], Y, A=A, logits_out=lg)
    return {"y": Y, "logits": lg}


def _quantize_plain(s):
    c = s["case"]
    x = s["x"] if s["rows"] is None else s["x"][s["rows"].long()]
    x = x.float()
    K, b = c["K"], BLOCK[c["fmt"]]
    if c["swiglu"]:
        x = _silu(x[:, :K]) * x[:, K:]
    pad = _padded(K) - K
    if pad:
        x = torch.cat([x, x.new_zeros(x.shape[0], pad)], 1)
    x = x.view(x.shape[0], -1, b)
    m = x.abs().amax(-1, keepdim=True)
    if c["fmt"] == "e4m3":
        d = (m / (6.0 * s["scale"])).clamp(max=448.0).to(torch.float8_e4m3fn).float() * s["scale"]
    else:  # the power of two at or below the largest value, two binades down
        e = (m.view(torch.int32) >> 23) - 2
        d = torch.where(m > 0, (e.clamp(min=1) << 23).view(torch.float32), torch.zeros_like(m))
    a, v = x.abs(), torch.zeros_like(x)
    v = v + 0.5 * (a > 0.25 * d) + 0.5 * (a >= 0.75 * d) + 0.5 * (a > 1.25 * d) + 0.5 * (a >= 1.75 * d)
    v = v + 1.0 * (a > 2.5 * d) + 1.0 * (a >= 3.5 * d) + 2.0 * (a > 5.0 * d)
    v = torch.where(x < 0, -v, v) * d
    return v.reshape(v.shape[0], -1)[:, :K].to(torch.bfloat16)


def _quantize_own(s):
    from routed_expert_ffn_topk_gb300 import estream as es
    c = s["case"]
    fmt = es.FP4_E4M3X16 if c["fmt"] == "e4m3" else es.FP4_E8M0X32
    q = es.mx4_quantize(s["x"], fmt, scale=s["scale"], rows=s["rows"], swiglu=c["swiglu"])
    return es.mx4_dequantize(q, torch.bfloat16)


def _values(codes, scales, fmt):
    """What codes and scale bytes stand for, in 32 bits."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2)
    d = scales.view(torch.float8_e4m3fn).float() if fmt == "e4m3" else torch.exp2(scales.float() - 127.0)
    return (v.unflatten(-1, (-1, BLOCK[fmt])) * d[..., None]).flatten(-2)


def _product_plain(s):
    c = s["case"]
    x, w = _values(*s["x"], c["fmt"]), _values(*s["w"], c["fmt"])
    if c["P"] == 1:
        y = x @ w[0].t()
    else:  # each slot's records, padded to the longest slot
        off, row = s["offsets"].long(), torch.arange(c["R"], device=x.device)
        slot = (row[:, None] >= off[None, 1:]).sum(1)
        at = row - off[slot]
        grid = torch.zeros(c["P"], s["cap"], x.shape[1], device=x.device)
        grid[slot, at] = x
        y = torch.bmm(grid, w.transpose(1, 2))[slot, at]
    return (y * (s["scale"][0] * s["scale"][1])).to(HALF[c["out"]])


def _product_own(s):
    from routed_expert_ffn_topk_gb300 import estream as es
    return es.mx4_product(s["x"], s["w"], offsets=s["offsets"], out_dtype=HALF[s["case"]["out"]])


def run(state):
    return {("decode", False): _layer_plain, ("decode", True): _layer_own, ("quantize", False): _quantize_plain,
            ("quantize", True): _quantize_own, ("product", False): _product_plain,
            ("product", True): _product_own}[state["case"]["op"], bool(own)](state)


def work(case):
    c = case
    if c["op"] == "decode":
        T, H, E, k, F, ns, Fs = (c[n] for n in ("T", "H", "E", "k", "F", "n_shared", "F_shared"))
        e = {"f32": 4.0, "bf16": 2.0, "q4": 9.0 / 16.0}[c["w"]]
        # experts that T tokens choose among, were the choices independent and even
        active = E * (1.0 - (1.0 - k / E) ** T)
        x = 4 if c["w"] == "f32" else 2
        b = 3 * H * e * (active * F + ns * Fs) + T * H * x + 4 * T * H * (1 if c["residual"] else 2)
        b += 2 * E * H + 4 * T * E if c["router"] else 4 * T * E
        return {"bytes": b, "flops": 6.0 * H * T * (k * F + ns * Fs) + (2.0 * T * E * H if c["router"] else 0.0)}
    if c["op"] == "quantize":  # the rows in, the codes and scales, and the values read back out of them
        R, K, b = c["R"], c["K"], BLOCK[c["fmt"]]
        n, w = c["src"] or R, K * (2 if c["swiglu"] else 1)
        q = R * (_padded(K) // 2 + _padded(K) // b)
        size = 4 if c["x"] == "f32" else 2
        return {"bytes": n * w * size + 2 * q + 2 * R * K + (4 * R if c["src"] else 0), "flops": 8.0 * R * K}
    R, N, K, P, b = c["R"], c["N"], c["K"], c["P"], BLOCK[c["fmt"]]
    row = _padded(K) // 2 + _padded(K) // b
    used = P * (1.0 - (1.0 - 1.0 / P) ** R) if P > 1 else 1
    return {"bytes": R * row + used * N * row + R * N * (4 if c["out"] == "f32" else 2), "flops": 2.0 * R * N * K}


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def _ffn64(x, wg, wu, wd):
    g, u = wg.double() @ x, wu.double() @ x
    return wd.double() @ (g / (1.0 + torch.exp(-g)) * u)


def _exact_layer(c, s):
    X = s["X"].double()
    lg = torch.einsum("th,eh->te", X, s["W_r"].double()) if c["router"] else s["logits"].double()
    out = X.clone() if c["residual"] else torch.zeros_like(X)
    for t in range(c["T"]):
        soft = torch.softmax(lg[t], 0)
        order = sorted(range(c["E"]), key=lambda e, v=lg[t].tolist(): (-v[e], e))[:c["k"]]
        total = sum(float(soft[e]) for e in order) if c["renorm"] else 1.0
        for e in order:
            out[t] += float(soft[e]) / total * _ffn64(X[t], *(w[e] for w in s["W"]))
        for j in range(c["n_shared"]):
            out[t] += _ffn64(X[t], *(w[j] for w in s["S"]))
    return {"y": out, "logits": lg} if c["router"] else {"y": out}


def _exact_quantize(c, s):
    x = s["x"].double()
    x = x if s["rows"] is None else x.index_select(0, s["rows"].long())
    if c["swiglu"]:
        gate, up = x.split(c["K"], 1)
        x = gate * torch.sigmoid(gate) * up
    R, K, b, g = c["R"], c["K"], BLOCK[c["fmt"]], s["scale"]
    levels = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    out = torch.empty_like(x)
    for r in range(0, R, 256):
        part = torch.nn.functional.pad(x[r:r + 256], (0, -K % b)).unflatten(1, (-1, b))
        top = part.abs().amax(2, keepdim=True)
        if c["fmt"] == "e4m3":  # to 4 significant bits, or to multiples of 2^-9 below 2^-6, ties to even
            want = (top / (6.0 * g)).clamp(max=448.0)
            ulp = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3.0)
            d = torch.round(want / ulp) * ulp * g
        else:
            d = torch.where(top > 0, torch.exp2((torch.frexp(top).exponent - 3).double()), torch.zeros_like(top))
        q = (part / torch.where(d > 0, d, torch.ones_like(d))).abs().clamp(max=6.0)
        step = torch.where(q < 2.0, 0.5, torch.where(q < 4.0, 1.0, 2.0)).double()
        q = torch.round(q / step) * step
        assert bool((levels[torch.searchsorted(levels, q)] == q).all())
        out[r:r + 256] = (torch.sign(part) * q * d).flatten(1)[:, :K]
    return out


def _exact_product(c, s):
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=DEV)

    def wide(codes, scales):
        d = scales.view(torch.float8_e4m3fn).double() if c["fmt"] == "e4m3" else torch.pow(2.0, scales.double() - 127)
        v = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=DEV)
        v[..., 0::2] = lut[codes.long() % 16]
        v[..., 1::2] = lut[codes.long() // 16]
        return v * d.repeat_interleave(BLOCK[c["fmt"]], -1)

    x = wide(*s["x"]) * s["scale"][0]
    out = torch.zeros(c["R"], c["N"], dtype=torch.float64, device=DEV)
    bounds = s["offsets"].tolist() if c["P"] > 1 else [0, c["R"]]
    for p in range(c["P"]):
        lo, hi = bounds[p], bounds[p + 1]
        if hi > lo:
            out[lo:hi] = x[lo:hi] @ (wide(s["w"][0][p], s["w"][1][p]) * s["scale"][1]).t()
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    with torch.no_grad():
        return {"decode": _exact_layer, "quantize": _exact_quantize, "product": _exact_product}[case["op"]](case, s)
