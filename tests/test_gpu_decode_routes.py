"""Routing inside the few-token layer call: the weights bit for bit, the router in
front past 128 experts, the largest route table, and what repeated calls share.

Tolerances are test_gpu_decode's."""
import numpy as np
import pytest
import torch

import oracle
from routed_expert_ffn_topk_gb300 import workloads as W
from tests import test_gpu_decode as D

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T", [1, 8, 9, 32])
@pytest.mark.parametrize("E,k", [(8, 2), (128, 8), (129, 6), (200, 32)])
def test_weights_bit_for_bit(E, k, T, renorm):
    """Expert e turns any token into 1 at column e of Y, exactly (SiLU(128) = 128 in
    fp32, times 1/128), so Y holds the tokens' weights: those of the written softmax."""
    wl = D._workload(T=T, H=256, E=E, k=k, F=128, renorm=renorm)
    lw = wl.layers[0]
    for t in (lw.Wg, lw.Wu, lw.Wd, wl.X):
        t.zero_()
    wl.X[:, 0] = 1.0
    lw.Wg[:, 0, 0] = 128.0
    lw.Wu[:, 0, 0] = 1.0 / 128
    lw.Wd[torch.arange(E), torch.arange(E), 0] = 1.0
    lg = wl.logits[0] * 4.0
    st = D._stack(wl)
    try:
        Y = torch.zeros(T, 256, device="cuda")
        st.decode(0, wl.X.cuda(), lg.cuda(), Y)
        D._ok(st)
        ids, alpha = oracle.route_topk(lg.numpy(), k, renorm)
        want = np.zeros((T, 256), np.float32)
        np.put_along_axis(want, np.asarray(ids).reshape(T, k).astype(np.int64),
                          np.asarray(alpha, dtype=np.float32).reshape(T, k), axis=1)
        np.testing.assert_array_equal(Y.cpu().numpy(), want)
    finally:
        st.close()


@pytest.mark.parametrize("w,T,E", [("bf16", 1, 129), ("bf16", 7, 200), ("q4", 3, 256), ("bf16", 32, 200), ("q4", 20, 160)])
def test_router_in_front_of_many_experts(w, T, E):
    wl = D._workload(T=T, H=512, E=E, k=5, F=128, w=w, n_shared=1, F_shared=256)
    wl.X, W_r = W.make_router(T, 512, E, seed=11)
    st = D._stack(wl, wdtype=D._dtype(w))
    try:
        lg = torch.empty(T, E, device="cuda")
        Y = torch.zeros(T, 512, device="cuda")
        st.poison()
        st.decode_from_x(0, wl.X.cuda(), W_r.cuda(), Y, logits_out=lg)
        D._ok(st)
        exact = wl.X.double() @ W_r.double().t()
        bound = (512 / 16 + 64) * 2.0 ** -24 * (wl.X.double().abs() @ W_r.double().abs().t())
        assert bool(((lg.cpu().double() - exact).abs() <= bound).all())
        D._check(Y.cpu(), D._reference(wl, w, logits=lg.cpu()), f"decode from X {w} T = {T} E = {E}")
    finally:
        st.close()


@pytest.mark.parametrize("w", ["bf16", "q4", "f32"])
def test_largest_route_table(w):
    """32 tokens with 32 routes each among 1024 experts, and shared experts: the
    table leaves the fewest stages for the weights' ring."""
    wl = D._workload(T=32, H=256, E=1024, k=32, F=128, w=w, n_shared=3, F_shared=256)
    st = D._stack(wl, wdtype=D._dtype(w))
    try:
        Y = torch.zeros(32, 256, device="cuda")
        st.decode(0, wl.X.cuda(), wl.logits[0].cuda(), Y)
        D._ok(st)
        D._check(Y.cpu(), D._reference(wl, w), f"decode, largest route table {w}")
    finally:
        st.close()


@pytest.mark.parametrize("w,T", [("bf16", 1), ("bf16", 8), ("bf16", 9), ("q4", 5), ("q4", 32), ("f32", 6)])
def test_calls_repeat_bit_for_bit(w, T):
    """The same call gives the same bits, with other calls in between; a row of a
    smaller batch agrees with the same token's row of the larger one to the sums'
    rounding (their order depends on the experts in use)."""
    wl = D._workload(T=T, H=512, E=24, k=4, F=256, w=w)
    st = D._stack(wl, wdtype=D._dtype(w))
    try:
        X, lg = wl.X.cuda(), wl.logits[0].cuda()
        ref = D._reference(wl, w)
        first = None
        for t in [T, 1, T, (T + 1) // 2, T]:
            Y = torch.zeros(t, 512, device="cuda")
            st.decode(0, X[:t], lg[:t], Y)
            D._ok(st)
            D._check(Y.cpu(), ref[:t], f"decode {w}, {t} of {T} tokens")
            if t == T:
                first = Y if first is None else first
                assert torch.equal(Y, first)
    finally:
        st.close()
