"""A prompt and the tokens after it through one MoE layer, on one GPU.

    python -m routed_expert_ffn_topk_gb300.generate --config c2 --batch 4 --prompt 256 --tokens 32
    python -m routed_expert_ffn_topk_gb300.generate --attention --temperature 0.8 --top-k 50 --top-p 0.95

The prompt goes through experts in microscaled 4-bit floating point (route map,
quantised gather, grouped product, SwiGLU quantised for the down product, weighted
sum); each generated token through the few-token layer call, one launch with the
router's logits formed in it, and then a dense 4-bit output projection. With
--attention the layer is preceded by attention over a paged key-value cache, which
the prompt fills and every token extends. Tokens are the likeliest ones, or drawn
from given random numbers. A token's step is captured once and replayed. Weights, embedding and projection are seeded
and random: it shows the calls together, not a language.
"""
from __future__ import annotations

import argparse
import math
import time

import torch

from . import estream as es
from . import workloads as W
from .layer import BoundLayerStack

# tensor scale of activations in E4M3X16: blocks with maxima from 0.0007 to 168 keep
# a scale of their own
ACT_SCALE = 2.0 ** -4


def mx4_weight_rows(w: torch.Tensor, fmt: int) -> es.Mx4Weights:
    """Weights [N, K] or [P, N, K] on the device, quantised for mx4_product."""
    rows = w.reshape(-1, w.shape[-1])
    q = es.mx4_quantize(rows, fmt, es.mx4_tensor_scale(float(rows.abs().max()), fmt))
    lead = tuple(w.shape[:-1])
    return es.mx4_weights(q.codes.view(*lead, -1), q.scales.view(*lead, -1), w.shape[-1], fmt, q.scale)


class Mx4Experts:
    """One layer's routed experts in 4 bits: Wg, Wu [E, F, H] and Wd [E, H, F]."""

    def __init__(self, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor, fmt: int = es.FP4_E4M3X16,
                 device="cuda"):
        self.fmt = fmt
        self.act_scale = ACT_SCALE if fmt == es.FP4_E4M3X16 else 1.0
        self.E, self.H = Wg.shape[0], Wg.shape[2]
        self.gate_up = mx4_weight_rows(torch.cat([Wg, Wu], 1).to(device), fmt)
        self.down = mx4_weight_rows(Wd.to(device), fmt)

    def prefill(self, X: torch.Tensor, logits: torch.Tensor, k: int, renorm: bool) -> torch.Tensor:
        """MoE(X) [T, H] in fp32; a token's routes are summed in rank order."""
        T = X.shape[0]
        if X.dim() != 2 or X.shape[1] != self.H or tuple(logits.shape) != (T, self.E):
            raise ValueError(f"X must be [T, {self.H}] and logits [T, {self.E}]")
        if T == 0:
            return torch.zeros(0, self.H, device=X.device)
        r = es.route_build(logits, k, renorm)
        offsets = r["offsets"][:self.E + 1]
        x = es.mx4_quantize(X, self.fmt, self.act_scale, rows=r["rec_tok"])
        gate_up = es.mx4_product(x, self.gate_up, offsets=offsets)
        h = es.mx4_quantize(gate_up, self.fmt, self.act_scale, swiglu=True)
        y = es.mx4_product(h, self.down, offsets=offsets, out_dtype=torch.float32)
        routes = torch.empty_like(y)
        routes[r["rec_route"].long()] = y  # from records to routes (t, rank)
        return (routes.view(T, k, self.H) * r["alpha"].view(T, k, 1)).sum(1)


class PagedAttention:
    """One attention layer of `batch` sequences of at most max_tokens: a 4-bit
    projection to queries, keys and values (Wqkv [(heads + 2 kv_heads) dim, H], queries
    first), keys and queries rotated by position, attention over the paged cache,
    and a 4-bit projection back (Wo [H, heads dim])."""

    def __init__(self, Wqkv: torch.Tensor, Wo: torch.Tensor, heads: int, kv_heads: int, batch: int, max_tokens: int,
                 page_size: int = 16, kv_dtype=torch.bfloat16, base: float = 10000.0, fmt: int = es.FP4_E4M3X16,
                 device="cuda"):
        self.heads, self.kv_heads, self.fmt, self.batch = heads, kv_heads, fmt, batch
        self.dim = Wqkv.shape[0] // (heads + 2 * kv_heads)
        self.act_scale = ACT_SCALE if fmt == es.FP4_E4M3X16 else 1.0
        self.qkv, self.out = mx4_weight_rows(Wqkv.to(device), fmt), mx4_weight_rows(Wo.to(device), fmt)
        M = -(-max_tokens // page_size)
        pages = torch.zeros(2, batch * M, page_size, kv_heads, self.dim, device=device).to(kv_dtype)
        self.cache = es.PagedKV(pages[0], pages[1])
        # an allocator hands pages out as sequences grow; here each has its own from the start
        self.table = torch.arange(batch * M, dtype=torch.int32, device=device).view(batch, M)
        self.max_tokens, self._lens = max_tokens, torch.zeros(batch, dtype=torch.int32, device=device)
        self._held = 0  # the longest sequence's tokens, as far as the host knows; None: ask the device
        self.inv_freq = (base ** (-torch.arange(0, self.dim, 2, dtype=torch.float64) / self.dim)).float().to(device)

    @property
    def lens(self) -> torch.Tensor:
        """The sequences' tokens, [batch] int32. A caller may set them (back, to give up tokens), asking for them here each time."""
        self._held = None
        return self._lens

    def reserve(self, n: int) -> int:
        """Refuses n more tokens than every sequence has room for; the longest one's tokens. The device is asked
        only where a caller may have changed the lengths, or before a refusal."""
        if self._held is None or self._held + n > self.max_tokens:
            self._held = int(self._lens.max())
        if self._held + n > self.max_tokens:
            raise ValueError(f"the attention layer holds {self.max_tokens} tokens a sequence: no room for {n} behind {self._held}")
        return self._held

    def _project(self, x: torch.Tensor, w: es.Mx4Weights) -> torch.Tensor:
        return es.mx4_product(es.mx4_quantize(x, self.fmt, self.act_scale), w)

    def _attend(self, X: torch.Tensor, positions: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                rows: torch.Tensor | None) -> torch.Tensor:
        qkv = self._project(X, self.qkv).view(X.shape[0], self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q = es.kv_append(self.cache, k, v, positions, self.table, rows=rows, q=q, inv_freq=self.inv_freq)
        a = es.kv_attend(self.cache, q, table, lens)
        return self._project(a.view(X.shape[0], -1), self.out)

    def prefill(self, X: torch.Tensor, m: int) -> torch.Tensor:
        """X [batch * m, H], m tokens of every sequence from its beginning: attention's output rows. Every
        token attends to itself and those before it: a row of its own length over its sequence's pages."""
        if not 1 <= m <= self.max_tokens or X.shape[0] != self.batch * m:
            raise ValueError(f"X must hold 1 to {self.max_tokens} tokens of {self.batch} sequences")
        positions = torch.arange(m, dtype=torch.int32, device=X.device).repeat(self.batch)
        rows = torch.arange(self.batch, dtype=torch.int32, device=X.device).repeat_interleave(m)
        y = self._attend(X, positions, positions + 1, self.table.repeat_interleave(m, 0), rows)
        self._lens.fill_(m)
        self._held = m
        return y

    def step(self, X: torch.Tensor) -> torch.Tensor:
        """X [batch, H], the next token of every sequence. Where it is captured, whoever replays it reserves the tokens."""
        held = None if torch.cuda.is_current_stream_capturing() else self.reserve(1)
        after = self._lens + 1
        y = self._attend(X, self._lens, after, self.table, None)
        self._lens.copy_(after)
        if held is not None:
            self._held = held + 1
        return y


class TokenLoop:
    """Tokens of up to DECODE_MAX_T sequences: embedding row [vocab, H], attention
    where there is one, layer with its residual, output projection [vocab, H], and
    the largest logit, or with `sampling` (sample_tokens' choices) a token drawn
    from a given random number."""

    def __init__(self, stack: BoundLayerStack, W_r: torch.Tensor, embedding: torch.Tensor, head: torch.Tensor,
                 fmt: int = es.FP4_E4M3X16, attention: PagedAttention | None = None, sampling: dict | None = None):
        self.stack, self.W_r, self.embedding, self.fmt = stack, W_r, embedding, fmt
        self.attention, self.sampling = attention, sampling
        self.head = mx4_weight_rows(head, fmt)
        self.act_scale = ACT_SCALE if fmt == es.FP4_E4M3X16 else 1.0
        self.graph = None

    def project(self, Y: torch.Tensor, u: torch.Tensor | None = None) -> torch.Tensor:
        """Token ids [n] of hidden rows [n, H], drawn from u [n] when sampling."""
        q = es.mx4_quantize(Y, self.fmt, self.act_scale)
        logits = es.mx4_product(q, self.head, out_dtype=torch.float32)
        if self.sampling is None:
            return logits.argmax(1)
        return es.sample_tokens(logits, u, **self.sampling).long()

    def attend(self, X: torch.Tensor, m: int | None = None) -> torch.Tensor:
        """X plus its attention, as rows of a prompt (m tokens a sequence) or as the next tokens."""
        if self.attention is None:
            return X
        return X + (self.attention.step(X) if m is None else self.attention.prefill(X, m))

    def step(self, ids: torch.Tensor, u: torch.Tensor | None = None) -> torch.Tensor:
        X = self.attend(self.embedding[ids])
        Y = torch.empty(X.shape, dtype=torch.float32, device=X.device)
        self.stack.decode_from_x(0, X, self.W_r, Y, residual=X)
        return self.project(Y, u)

    def numbers(self, u: torch.Tensor | None, n: int, b: int) -> torch.Tensor | None:
        """The random numbers of n tokens of b sequences: u [n, b] when sampling, else none."""
        if self.sampling is None:
            return None
        if not isinstance(u, torch.Tensor) or tuple(u.shape) != (n, b):
            raise ValueError(f"sampling needs random numbers [{n}, {b}]")
        return u

    def _as_captured(self, ids: torch.Tensor) -> bool:
        """Whether the captured step is for as many sequences and the present choices."""
        if self.graph is None or self.ids.shape != ids.shape or (self.choices is None) != (self.sampling is None):
            return False
        same = lambda x, y: x is y or not (torch.is_tensor(x) or torch.is_tensor(y)) and x == y
        return self.choices is None or (self.choices.keys() == self.sampling.keys()
                                        and all(same(x, self.sampling[k]) for k, x in self.choices.items()))

    def run(self, ids: torch.Tensor, n: int, u: torch.Tensor | None = None) -> torch.Tensor:
        """The n tokens after ids [b] of every sequence, [b, n]; u [n, b] random numbers when sampling."""
        u = self.numbers(u, n, ids.shape[0])
        held = None if self.attention is None else self.attention.reserve(n)
        if n == 0:
            return ids[:, None][:, :0]
        if not self._as_captured(ids):
            self.ids, self.choices = ids.clone(), None if self.sampling is None else dict(self.sampling)
            self.u = None if u is None else torch.zeros(ids.shape, dtype=torch.float32, device=ids.device)
            lens = None if self.attention is None else self.attention._lens.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self.step(self.ids, self.u)  # allocations and first-call work outside the capture
            torch.cuda.current_stream().wait_stream(side)
            if lens is not None:
                self.attention._lens.copy_(lens)  # the next step stores its token in that one's place
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.ids.copy_(self.step(self.ids, self.u))
        if held is not None:
            self.attention._held = None  # until all n are held
        self.ids.copy_(ids)
        out = torch.empty(ids.shape[0], n, dtype=ids.dtype, device=ids.device)
        for i in range(n):
            if u is not None:
                self.u.copy_(u[i])
            self.graph.replay()
            out[:, i] = self.ids
        if held is not None:
            self.attention._held = held + n
        return out


def build(config: str, batch: int, vocab: int, seed: int = 0, wdtype=None, attend_tokens: int = 0,
          sampling: dict | None = None):
    """The layer of a workload configuration with an embedding and a router, and with attend_tokens
    an attention layer (heads of 128, a key head for four of them) for sequences of as many tokens."""
    import dataclasses

    cfg = dataclasses.replace(W.CONFIGS[config], T=batch)
    wl = W.make_workload(cfg)
    g = torch.Generator().manual_seed(seed)
    emb, head = (torch.randn(vocab, cfg.H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    W_r = (torch.randn(cfg.E, cfg.H, generator=g) / math.sqrt(cfg.H)).to(torch.bfloat16).cuda()
    lw = wl.layers[0]
    experts = Mx4Experts(lw.Wg, lw.Wu, lw.Wd)
    stack = BoundLayerStack(wl, mode="resident", wdtype=wdtype)
    attention = None
    if attend_tokens:
        heads, dim = max(1, cfg.H // 128), min(cfg.H, 128)
        kv_heads = max(1, heads // 4)
        Wqkv = torch.randn((heads + 2 * kv_heads) * dim, cfg.H, generator=g) / math.sqrt(cfg.H)
        Wo = torch.randn(cfg.H, heads * dim, generator=g) / math.sqrt(heads * dim)
        attention = PagedAttention(Wqkv.to(torch.bfloat16), Wo.to(torch.bfloat16), heads, kv_heads, batch, attend_tokens)
    return cfg, experts, TokenLoop(stack, W_r, emb, head, attention=attention, sampling=sampling)


def generate(cfg, experts: Mx4Experts, loop: TokenLoop, prompt: torch.Tensor, n: int,
             u: torch.Tensor | None = None) -> torch.Tensor:
    """prompt [b, m] token ids; the n tokens after it, [b, n]; u [n, b] random numbers when sampling."""
    if loop.attention is not None and prompt.shape[1] + n - 1 > loop.attention.max_tokens:
        raise ValueError(f"the attention layer holds {loop.attention.max_tokens} tokens a sequence")
    u = loop.numbers(u, n, prompt.shape[0])
    X = loop.attend(loop.embedding[prompt.reshape(-1)], prompt.shape[1])
    logits = es.router_logits(X, loop.W_r)
    Y = X.float() + experts.prefill(X, logits, cfg.k, cfg.renorm)
    first = loop.project(Y.view(*prompt.shape, cfg.H)[:, -1], None if u is None else u[0])
    rest = loop.run(first, n - 1, None if u is None else u[1:]) if n > 1 else first[:, None][:, :0]
    return torch.cat([first[:, None], rest], 1)


def main() -> None:
    p = argparse.ArgumentParser(description="a prompt and its next tokens through one MoE layer")
    p.add_argument("--config", default="c2", help="a layer configuration without shared experts, bf16")
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--prompt", type=int, default=256)
    p.add_argument("--tokens", type=int, default=32)
    p.add_argument("--vocab", type=int, default=8192)
    p.add_argument("--attention", action="store_true", help="attention over a paged cache before the layer")
    p.add_argument("--temperature", type=float, default=0.0, help="0: the likeliest token")
    p.add_argument("--top-k", type=int, default=0)
    p.add_argument("--top-p", type=float, default=1.0)
    p.add_argument("--min-p", type=float, default=0.0)
    a = p.parse_args()
    c = W.CONFIGS[a.config]
    if c.dtype != "bf16" or c.n_shared:
        p.error("the configuration must be bf16 and without shared experts")
    if not 1 <= a.batch <= es.DECODE_MAX_T or min(a.prompt, a.tokens, a.vocab) < 1:
        p.error(f"1 to {es.DECODE_MAX_T} sequences, and at least one token of prompt and output")
    sampling = None
    if a.temperature > 0:
        sampling = dict(temperature=a.temperature, top_k=a.top_k, top_p=a.top_p, min_p=a.min_p)
    cfg, experts, loop = build(a.config, a.batch, a.vocab, sampling=sampling,
                               attend_tokens=a.prompt + a.tokens if a.attention else 0)
    g = torch.Generator().manual_seed(1)
    prompt = torch.randint(0, a.vocab, (a.batch, a.prompt), generator=g).cuda()
    u = torch.rand(a.tokens, a.batch, generator=g).cuda() if sampling else None
    generate(cfg, experts, loop, prompt, a.tokens, u)  # first-call work
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    ids = generate(cfg, experts, loop, prompt, a.tokens, u)
    torch.cuda.synchronize()
    t = time.perf_counter() - t0
    if es.get_device_error(loop.stack.ctx) != es.OK or es.mx4_error() != es.OK:
        raise RuntimeError("device error")
    print(f"{a.batch} sequences, {a.prompt} prompt tokens and {a.tokens} generated each: {t * 1e3:.2f} ms")
    print(ids[0].tolist())


if __name__ == "__main__":
    main()
