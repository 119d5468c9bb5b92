"""A prompt and the tokens after it through one MoE layer, on one GPU.

    python -m routed_expert_ffn_topk_gb300.generate --config c2 --batch 4 --prompt 256 --tokens 32

The prompt goes through experts in microscaled 4-bit floating point (route map,
quantised gather, grouped product, SwiGLU quantised for the down product, weighted
sum); each generated token through the few-token layer call, one launch with the
router's logits formed in it, and then a dense 4-bit output projection. A token's
step is captured once and replayed. Weights, embedding and projection are seeded
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


class TokenLoop:
    """Greedy tokens of up to DECODE_MAX_T sequences: embedding row [vocab, H], layer
    with its residual, output projection [vocab, H], largest logit."""

    def __init__(self, stack: BoundLayerStack, W_r: torch.Tensor, embedding: torch.Tensor, head: torch.Tensor,
                 fmt: int = es.FP4_E4M3X16):
        self.stack, self.W_r, self.embedding, self.fmt = stack, W_r, embedding, fmt
        self.head = mx4_weight_rows(head, fmt)
        self.act_scale = ACT_SCALE if fmt == es.FP4_E4M3X16 else 1.0
        self.graph = None

    def project(self, Y: torch.Tensor) -> torch.Tensor:
        """Token ids [n] of hidden rows [n, H]."""
        q = es.mx4_quantize(Y, self.fmt, self.act_scale)
        return es.mx4_product(q, self.head, out_dtype=torch.float32).argmax(1)

    def step(self, ids: torch.Tensor) -> torch.Tensor:
        X = self.embedding[ids]
        Y = torch.empty(X.shape, dtype=torch.float32, device=X.device)
        self.stack.decode_from_x(0, X, self.W_r, Y, residual=X)
        return self.project(Y)

    def run(self, ids: torch.Tensor, n: int) -> torch.Tensor:
        """The n tokens after ids [b] of every sequence, [b, n]."""
        if self.graph is None or self.ids.shape != ids.shape:
            self.ids = ids.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                self.step(self.ids)  # allocations and first-call work outside the capture
            torch.cuda.current_stream().wait_stream(side)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.ids.copy_(self.step(self.ids))
        self.ids.copy_(ids)
        out = torch.empty(ids.shape[0], n, dtype=ids.dtype, device=ids.device)
        for i in range(n):
            self.graph.replay()
            out[:, i] = self.ids
        return out


def build(config: str, batch: int, vocab: int, seed: int = 0, wdtype=None):
    """The layer of a workload configuration with an embedding and a router."""
    import dataclasses

    cfg = dataclasses.replace(W.CONFIGS[config], T=batch)
    wl = W.make_workload(cfg)
    g = torch.Generator().manual_seed(seed)
    emb, head = (torch.randn(vocab, cfg.H, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    W_r = (torch.randn(cfg.E, cfg.H, generator=g) / math.sqrt(cfg.H)).to(torch.bfloat16).cuda()
    lw = wl.layers[0]
    experts = Mx4Experts(lw.Wg, lw.Wu, lw.Wd)
    stack = BoundLayerStack(wl, mode="resident", wdtype=wdtype)
    return cfg, experts, TokenLoop(stack, W_r, emb, head)


def generate(cfg, experts: Mx4Experts, loop: TokenLoop, prompt: torch.Tensor, n: int) -> torch.Tensor:
    """prompt [b, m] token ids; the n tokens after it, [b, n]."""
    X = loop.embedding[prompt.reshape(-1)]
    logits = es.router_logits(X, loop.W_r)
    Y = X.float() + experts.prefill(X, logits, cfg.k, cfg.renorm)
    first = loop.project(Y.view(*prompt.shape, cfg.H)[:, -1])
    rest = loop.run(first, n - 1) if n > 1 else first[:, None][:, :0]
    return torch.cat([first[:, None], rest], 1)


def main() -> None:
    p = argparse.ArgumentParser(description="a prompt and its next tokens through one MoE layer")
    p.add_argument("--config", default="c2", help="a layer configuration without shared experts, bf16")
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--prompt", type=int, default=256)
    p.add_argument("--tokens", type=int, default=32)
    p.add_argument("--vocab", type=int, default=8192)
    a = p.parse_args()
    c = W.CONFIGS[a.config]
    if c.dtype != "bf16" or c.n_shared:
        p.error("the configuration must be bf16 and without shared experts")
    if not 1 <= a.batch <= es.DECODE_MAX_T or min(a.prompt, a.tokens, a.vocab) < 1:
        p.error(f"1 to {es.DECODE_MAX_T} sequences, and at least one token of prompt and output")
    cfg, experts, loop = build(a.config, a.batch, a.vocab)
    prompt = torch.randint(0, a.vocab, (a.batch, a.prompt), generator=torch.Generator().manual_seed(1)).cuda()
    generate(cfg, experts, loop, prompt, a.tokens)  # first-call work
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    ids = generate(cfg, experts, loop, prompt, a.tokens)
    torch.cuda.synchronize()
    t = time.perf_counter() - t0
    if es.get_device_error(loop.stack.ctx) != es.OK or es.mx4_error() != es.OK:
        raise RuntimeError("device error")
    print(f"{a.batch} sequences, {a.prompt} prompt tokens and {a.tokens} generated each: {t * 1e3:.2f} ms")
    print(ids[0].tolist())


if __name__ == "__main__":
    main()
