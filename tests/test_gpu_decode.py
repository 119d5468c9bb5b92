"""The few-token layer call (estream_moe_layer_decode, ..._from_x) against the
fp64 oracle.

Tolerance: every product is of exactly represented operands and every sum is in
fp32. A sum of n terms of random sign carries a relative error of about
sqrt(n) 2^-24 (twice that where the tensor cores truncate), at most 1.5e-5 for
the longest sums here (n = 14336); Y goes through two such sums, so the 2-norm of
the error over the 2-norm of the layer's output stays below REL = 2e-5. A token's
alpha is bit-exact. Results are also held to the layer tests' own bounds."""
import numpy as np
import pytest
import torch

import oracle
from routed_expert_ffn_topk_gb300 import workloads as W
from tests import _gpu

pytestmark = pytest.mark.gpu

REL = 2e-5


def _es():
    from routed_expert_ffn_topk_gb300 import estream as es
    return es


def _stack(wl, **kw):
    from routed_expert_ffn_topk_gb300.layer import BoundLayerStack
    return BoundLayerStack(wl, mode="resident", **kw)


def _dtype(name):
    es = _es()
    return {"bf16": es.BF16, "q4": es.Q4, "f32": es.F32}[name]


def _workload(T, H, E, k, F, w="bf16", renorm=False, n_shared=0, F_shared=0, seed=5):
    base = W.CONFIGS["c1" if w == "f32" else "c2"]
    import dataclasses
    cfg = dataclasses.replace(base, key="dec", T=T, H=H, E=E, k=k, F=F, renorm=renorm, n_shared=n_shared,
                              F_shared=F_shared, G=min(base.G, E), B=1, P=min(base.G, E), x_std=1.0)
    return W.make_workload(cfg, seed=seed)


def _reference(wl, w, X=None, logits=None):
    cfg = wl.cfg
    X = wl.X if X is None else X
    lw = wl.layers[0]
    lg = wl.logits[0] if logits is None else logits
    ids, alpha = oracle.route_topk(lg.numpy(), cfg.k, cfg.renorm)
    if w == "q4":
        Wg, Wu, Wd, shared = _gpu.q4_weights(lw)
        return oracle.moe_layer_rows(X.float().numpy(), Wg, Wu, Wd, ids, alpha, shared=shared)
    shared = (lw.Sg, lw.Su, lw.Sd) if cfg.n_shared else None
    return oracle.moe_layer_rows(X, lw.Wg, lw.Wu, lw.Wd, ids, alpha, shared=shared)


def _check(y, ref, what):
    y = np.asarray(y, dtype=np.float64)
    _gpu.assert_y_close(y, ref, what)
    rel = np.linalg.norm(y - ref) / np.linalg.norm(ref)
    assert rel <= REL, f"{what}: {rel:.2e}"


def _ok(st):
    torch.cuda.synchronize()
    assert _es().get_device_error(st.ctx) == _es().OK


SHAPES = {
    "one_token": dict(T=1, H=512, E=16, k=4, F=256),
    "two_tokens_one_expert_each": dict(T=2, H=256, E=8, k=1, F=128),
    "seven": dict(T=7, H=768, E=12, k=3, F=384),
    "eight": dict(T=8, H=512, E=16, k=4, F=256),
    "nine": dict(T=9, H=512, E=5, k=5, F=640),
    "thirty_two": dict(T=32, H=1024, E=64, k=8, F=512),
    "one_expert": dict(T=32, H=256, E=1, k=1, F=128),
    "seventeen_renorm": dict(T=17, H=256, E=40, k=6, F=1408, renorm=True),
    "shared": dict(T=5, H=512, E=8, k=2, F=256, renorm=True, n_shared=2, F_shared=384),
    "shared_wide_32": dict(T=32, H=256, E=8, k=2, F=256, n_shared=1, F_shared=1152),
    "all_experts": dict(T=3, H=256, E=32, k=32, F=128),
    "max_experts": dict(T=4, H=256, E=1024, k=32, F=128),
    "wide": dict(T=2, H=4096, E=2, k=2, F=1024),
}


@pytest.mark.parametrize("w", ["bf16", "q4", "f32"])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_layer(shape, w):
    """Y += MoE(X), and the same bit for bit again; then Y = A + MoE(X)."""
    wl = _workload(w=w, **SHAPES[shape])
    st = _stack(wl, wdtype=_dtype(w))
    try:
        X, lg = wl.X.cuda(), wl.logits[0].cuda()
        ys = []
        for _ in range(2):
            st.poison()
            Y = torch.zeros(wl.cfg.T, wl.cfg.H, device="cuda")
            st.decode(0, X, lg, Y)
            ys.append(Y)
        _ok(st)
        ref = _reference(wl, w)
        _check(ys[0].cpu(), ref, f"decode {shape}/{w}")
        assert torch.equal(ys[0], ys[1])
        A = (torch.randn(wl.cfg.T, wl.cfg.H, generator=torch.Generator().manual_seed(1)) * 0.1).to(X.dtype)
        Y = torch.full_like(ys[0], float("nan"))
        st.decode(0, X, lg, Y, residual=A.cuda())
        _ok(st)
        _check(Y.cpu(), ref + A.double().numpy(), f"decode {shape}/{w} + A")
        Y = A.float().cuda()
        st.decode(0, X, lg, Y)
        _ok(st)
        _check(Y.cpu(), ref + A.double().numpy(), f"decode {shape}/{w} into Y")
    finally:
        st.close()


@pytest.mark.parametrize("T", [1, 8, 32])
def test_every_token_count_on_one_context(T):
    """Prefixes of one batch give the same rows bit for bit: a token's row does
    not depend on the other tokens of the call."""
    wl = _workload(T=32, H=512, E=24, k=4, F=256)
    st = _stack(wl)
    try:
        X, lg = wl.X.cuda(), wl.logits[0].cuda()
        ref = _reference(wl, "bf16")
        for t in range(1, T + 1, 3):
            Y = torch.zeros(t, 512, device="cuda")
            st.decode(0, X[:t], lg[:t], Y)
            _ok(st)
            _check(Y.cpu(), ref[:t], f"decode T = {t}")
    finally:
        st.close()


@pytest.mark.parametrize("w", ["bf16", "q4"])
def test_storage_order_and_groups(w):
    """Experts in another storage order, in groups that do not divide E."""
    wl = _workload(T=6, H=256, E=11, k=3, F=256, w=w)
    st = _stack(wl, wdtype=_dtype(w), G=4, perm=W.random_permutation(11, 3).reshape(1, -1))
    try:
        Y = torch.zeros(6, 256, device="cuda")
        st.decode(0, wl.X.cuda(), wl.logits[0].cuda(), Y)
        _ok(st)
        _check(Y.cpu(), _reference(wl, w), f"decode storage order {w}")
    finally:
        st.close()


def test_ties_take_the_lower_expert():
    wl = _workload(T=4, H=256, E=16, k=3, F=128)
    wl.logits[0] = torch.zeros(4, 16)
    wl.logits[0][1, 5] = 1.0
    wl.logits[0][2] = -0.0
    wl.logits[0][3, 9:] = float("-inf")
    st = _stack(wl)
    try:
        Y = torch.zeros(4, 256, device="cuda")
        st.decode(0, wl.X.cuda(), wl.logits[0].cuda(), Y)
        _ok(st)
        _check(Y.cpu(), _reference(wl, "bf16"), "decode ties")
    finally:
        st.close()


@pytest.mark.parametrize("w,T", [("bf16", 1), ("bf16", 5), ("q4", 3), ("bf16", 32)])
def test_from_x(w, T):
    """Router logits within the fp32 summation bound of the fp64 ones, and the
    layer of those logits."""
    wl = _workload(T=T, H=1024, E=60, k=4, F=256, w=w, n_shared=1, F_shared=256)
    X, W_r = W.make_router(T, 1024, 60, seed=11)
    wl.X = X
    st = _stack(wl, wdtype=_dtype(w))
    try:
        lg = torch.empty(T, 60, device="cuda")
        Y = torch.zeros(T, 1024, device="cuda")
        st.poison()
        st.decode_from_x(0, X.cuda(), W_r.cuda(), Y, logits_out=lg)
        _ok(st)
        exact = X.double() @ W_r.double().t()
        bound = (1024 / 16 + 64) * 2.0 ** -24 * (X.double().abs() @ W_r.double().abs().t())
        assert bool(((lg.cpu().double() - exact).abs() <= bound).all())
        _check(Y.cpu(), _reference(wl, w, logits=lg.cpu()), f"decode from X {w} T = {T}")
        Y2 = torch.zeros_like(Y)
        st.decode_from_x(0, X.cuda(), W_r.cuda(), Y2)          # logits kept inside
        st.decode(0, X.cuda(), lg, Y)                          # accumulates
        _ok(st)
        assert torch.equal(2 * Y2, Y)
    finally:
        st.close()


def test_same_as_the_prompt_call():
    """The prompt and the generation call read one arena; they agree to the
    prompt call's accuracy (fp16 h)."""
    wl = _workload(T=16, H=512, E=16, k=4, F=256, n_shared=1, F_shared=256)
    st = _stack(wl)
    try:
        X, lg = wl.X.cuda(), wl.logits[0].cuda()
        Y, P = torch.zeros(16, 512, device="cuda"), torch.zeros(16, 512, device="cuda")
        st.prefill(0, X, lg, P)
        st.decode(0, X, lg, Y)
        st.prefill(0, X, lg, P)
        _ok(st)
        _gpu.assert_y_close(P.cpu().numpy() / 2, Y.cpu().numpy(), "prompt call against generation call")
    finally:
        st.close()


def test_non_finite_and_large_activations():
    """A NaN or infinity stays in its token's row; an h beyond fp16's range is
    computed (the prompt call reports it as an error)."""
    wl = _workload(T=4, H=256, E=8, k=2, F=256)
    X = wl.X.clone()
    X[3, :4] = 2.0 ** 14
    st = _stack(wl)
    try:
        ref = _reference(wl, "bf16", X=X)
        bad = X.clone()
        bad[0, 7] = float("nan")
        bad[2, 9] = float("inf")
        Y = torch.zeros(4, 256, device="cuda")
        st.decode(0, bad.cuda(), wl.logits[0].cuda(), Y)
        _ok(st)
        y = Y.cpu().numpy()
        assert np.isnan(y[0]).all() and not np.isfinite(y[2]).any()
        _check(y[[1]], ref[[1]], "beside a NaN")
        _check(y[[3]], ref[[3]], "large h")
    finally:
        st.close()


@pytest.mark.parametrize("w", ["bf16", "q4", "f32"])
def test_graph_replay_and_streams(w):
    """Captured into a CUDA graph and replayed on new inputs, and called on a side
    stream: bit-identical to the plain call."""
    wl = _workload(T=3, H=256, E=8, k=2, F=256, w=w)
    st = _stack(wl, wdtype=_dtype(w))
    try:
        X, lg = wl.X.cuda(), wl.logits[0].cuda()
        X2, lg2 = (X * 0.5).clone(), lg.flip(1).contiguous()
        want = []
        for x, l in ((X, lg), (X2, lg2)):
            Y = torch.empty(3, 256, device="cuda")
            st.decode(0, x, l, Y, residual=x)
            want.append(Y)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = torch.empty(3, 256, device="cuda")
        st.decode(0, X2, lg2, got, residual=X2, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        _ok(st)
        assert torch.equal(got, want[1])
        bx, bl, by = X.clone(), lg.clone(), torch.empty(3, 256, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st.decode(0, bx, bl, by, residual=bx)
        for x, l, y in ((X2, lg2, want[1]), (X, lg, want[0])):
            bx.copy_(x)
            bl.copy_(l)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(by, y)
    finally:
        st.close()


def test_barriers_give_up():
    """One CTA withholds its arrival: the others' bounded wait runs out, the call
    reports it and leaves Y alone, and the next call is normal."""
    es = _es()
    wl = _workload(T=2, H=256, E=8, k=2, F=128)
    X, W_r = W.make_router(2, 256, 8, seed=3)
    wl.X = X
    st = _stack(wl)
    try:
        X, W_r = X.cuda(), W_r.cuda()
        want = torch.zeros(2, 256, device="cuda")
        st.decode_from_x(0, X, W_r, want)
        _ok(st)
        for inject in (es.inject_expert_timeout, es.inject_route_timeout):
            inject(st.ctx)
            Y = torch.full((2, 256), 7.0, device="cuda")
            st.decode_from_x(0, X, W_r, Y)
            torch.cuda.synchronize()
            assert es.get_device_error(st.ctx) == es.ERR_TIMEOUT
            assert bool((Y == 7.0).all())
            Y = torch.zeros(2, 256, device="cuda")
            st.decode_from_x(0, X, W_r, Y)
            _ok(st)
            assert torch.equal(Y, want)
    finally:
        st.close()


def test_full_size_shapes():
    """One and a few tokens through the full-size layers' weights."""
    import dataclasses
    for key, T in (("c2", 1), ("c2", 16), ("c3", 4)):
        cfg = dataclasses.replace(W.CONFIGS[key], T=T)
        wl = W.make_workload(cfg)
        st = _stack(wl)
        try:
            Y = torch.zeros(T, cfg.H, device="cuda")
            st.decode(0, wl.X.cuda(), wl.logits[0].cuda(), Y)
            _ok(st)
            _check(Y.cpu(), _reference(wl, "bf16"), f"decode {key} T = {T}")
        finally:
            st.close()


def test_refusals():
    es = _es()
    wl = _workload(T=33, H=256, E=8, k=2, F=128)
    X, lg = wl.X.cuda(), wl.logits[0].cuda()
    Y = torch.zeros(33, 256, device="cuda")
    W_r = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")

    def status(fn):
        with pytest.raises(es.EStreamError) as e:
            fn()
        return e.value.status

    st = _stack(wl)
    try:
        assert status(lambda: st.decode(0, X, lg, Y)) == es.ERR_CAPACITY                    # T = 33
        assert status(lambda: st.decode(0, X[:2], lg[:2], Y[:2], k=3)) == es.ERR_CAPACITY   # k > k_max
        assert status(lambda: st.decode(0, X[:2], lg[:2], Y[:2], k=9)) == es.ERR_INVALID_ARG
        assert status(lambda: st.decode(1, X[:2], lg[:2], Y[:2])) == es.ERR_INVALID_ARG     # layer
        with pytest.raises(ValueError):
            st.decode(0, X[:2].float(), lg[:2], Y[:2])
        with pytest.raises(ValueError):
            st.decode(0, X[:2], lg[:3], Y[:2])
        with pytest.raises(ValueError):
            st.decode(0, X[:2], lg[:2, :7], Y[:2])
        with pytest.raises(ValueError):
            st.decode_from_x(0, X[:2], W_r[:7], Y[:2])
        with pytest.raises(ValueError):
            st.decode_from_x(0, X[:2], W_r, Y[:2], logits_out=torch.empty(2, 7, device="cuda"))
        es.arena_invalidate(st.ctx)
        assert status(lambda: st.decode(0, X[:2], lg[:2], Y[:2])) == es.ERR_CAPACITY        # not resident
        es.arena_preload(st.ctx, 0)
        st.decode(0, X[:2], lg[:2], Y[:2])
        _ok(st)
    finally:
        st.close()
    wl = _workload(T=2, H=256, E=8, k=2, F=128, w="f32")
    st = _stack(wl)
    try:
        s = es.lib().estream_moe_layer_decode_from_x(st.ctx, 0, X.data_ptr(), W_r.data_ptr(), 2, 2, 0, None,
                                                     Y.data_ptr(), None, None)
        assert s == es.ERR_INVALID_ARG
    finally:
        st.close()
