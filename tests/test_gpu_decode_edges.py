"""The few-token layer call where things leave the ordinary: non-finite weights and logits,
largest activations, late arrivals at its grid barriers, calls on streams that nothing orders.

Tolerances are test_gpu_decode's."""
import numpy as np
import pytest
import torch

from tests import test_gpu_decode as D

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("w", ["bf16", "q4", "f32"])
@pytest.mark.parametrize("T", [1, 2, 8, 9])
def test_non_finite_down_weight_stays_with_its_expert(T, w, value):
    """Expert 3 has an infinite or NaN down weight. A token that takes it has a
    non-finite value in that row of Y; the other tokens' rows are what they are
    without it."""
    if w == "q4" and np.isnan(value):
        pytest.skip("4-bit codes hold no NaN")
    wl = D._workload(T=T, H=256, E=8, k=2, F=256, w=w)
    lg = wl.logits[0]
    lg[:, 3] = -50.0          # nobody's
    if T > 1:
        lg[T - 1, 3] = 50.0   # but the last token's
    ref = D._reference(wl, w)
    wl.layers[0].Wd[3, 17, 40] = value
    st = D._stack(wl, wdtype=D._dtype(w))
    try:
        Y = torch.zeros(T, 256, device="cuda")
        st.decode(0, wl.X.cuda(), lg.cuda(), Y)
        D._ok(st)
        y = Y.cpu().numpy()
        others = slice(0, T - 1 if T > 1 else 1)
        D._check(y[others], ref[others], f"beside a non-finite weight {w} T = {T}")
        if T > 1:
            assert not np.isfinite(y[T - 1, 17])
    finally:
        st.close()


@pytest.mark.parametrize("w,T,barrier", [("bf16", 2, 0), ("bf16", 2, 1), ("q4", 3, 1), ("f32", 2, 1), ("bf16", 12, 0),
                                         ("bf16", 12, 1), ("bf16", 12, 2), ("q4", 12, 2)])
def test_late_arrival_leaves_y(w, T, barrier):
    """A CTA that arrives at a grid barrier after the others gave up does not go on
    alone: Y, accumulated into here, stays as it was, and the next call is normal."""
    es = D._es()
    wl = D._workload(T=T, H=256, E=8, k=2, F=128, w=w)
    W_r = None
    if w != "f32":
        wl.X, W_r = D.W.make_router(T, 256, 8, seed=3)
    st = D._stack(wl, wdtype=D._dtype(w))

    def call(Y):
        if W_r is None:
            st.decode(0, X, wl.logits[0].cuda(), Y)
        else:
            st.decode_from_x(0, X, W_r, Y)

    try:
        X = wl.X.cuda()
        W_r = None if W_r is None else W_r.cuda()
        want = torch.zeros(T, 256, device="cuda")
        call(want)
        D._ok(st)
        es.inject_late_arrival(st.ctx, barrier)
        Y = torch.full((T, 256), 7.0, device="cuda")
        call(Y)
        torch.cuda.synchronize()
        assert es.get_device_error(st.ctx) == es.ERR_TIMEOUT
        assert bool((Y == 7.0).all())
        Y = torch.zeros(T, 256, device="cuda")
        call(Y)
        D._ok(st)
        assert torch.equal(Y, want)
        with pytest.raises(es.EStreamError):
            es.inject_late_arrival(st.ctx, 3)
    finally:
        st.close()


@pytest.mark.parametrize("w,T", [("f32", 4), ("bf16", 3), ("bf16", 20), ("q4", 5)])
def test_streams_without_an_order(w, T):
    """Calls on two streams that nothing orders, as fast as they can be made: each
    has the result that it has alone."""
    wl = D._workload(T=T, H=512, E=16, k=4, F=512, w=w)
    st = D._stack(wl, wdtype=D._dtype(w))
    try:
        lg = wl.logits[0].cuda()
        Xs = [wl.X.cuda(), (wl.X * 0.5).cuda(), wl.X.flip(0).contiguous().cuda()]
        want = []
        for X in Xs:
            Y = torch.zeros(T, 512, device="cuda")
            st.decode(0, X, lg, Y)
            want.append(Y)
        D._ok(st)
        streams = [torch.cuda.Stream() for _ in range(3)]
        Ys = torch.zeros(300, T, 512, device="cuda")
        torch.cuda.synchronize()
        for i in range(300):
            st.decode(0, Xs[i % 3], lg, Ys[i], stream=streams[i % 3])
        D._ok(st)
        for i in range(300):
            assert torch.equal(Ys[i], want[i % 3]), i
    finally:
        st.close()


@pytest.mark.parametrize("w", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 9])
@pytest.mark.parametrize("E", [8, 128, 130, 200])
def test_nan_logits(E, T, w):
    """A NaN among a token's logits makes its softmax, and with it its row of Y, NaN
    in either form of the selection; the other rows are what they are without it."""
    wl = D._workload(T=T, H=256, E=E, k=2, F=128, w=w)
    ref = D._reference(wl, w)
    others = [t for t in range(T) if t != 1]
    st = D._stack(wl, wdtype=D._dtype(w))
    try:
        for bits in (0x7fc00000, 0xffc00000, 0xffffffff):
            for where in (slice(None), slice(5, 6)):
                lg = wl.logits[0].numpy().copy()
                lg.view(np.uint32)[1, where] = bits
                Y = torch.zeros(T, 256, device="cuda")
                st.decode(0, wl.X.cuda(), torch.from_numpy(lg).cuda(), Y)
                D._ok(st)
                y = Y.cpu().numpy()
                assert np.isnan(y[1]).all()
                D._check(y[others], ref[others], f"beside NaN logits {w} E = {E} T = {T}")
    finally:
        st.close()


@pytest.mark.parametrize("infinite", [False, True])
@pytest.mark.parametrize("T", [1, 9])
def test_h_at_the_top_of_the_range(T, infinite):
    """h = (181 / 128)^2 2^127, which bf16 rounds to infinity: Y, a thousandth of it,
    is exact. An infinite h gives an infinite Y."""
    wl = D._workload(T=T, H=256, E=1, k=1, F=128)
    lw = wl.layers[0]
    for t in (lw.Wg, lw.Wu, lw.Wd, wl.X):
        t.zero_()
    wl.X[:, 0] = 2.0 ** 32
    lw.Wg[0, 0, 0] = 181 / 128 * 2.0 ** (40 if infinite else 31)  # SiLU of so much is itself
    lw.Wu[0, 0, 0] = 181 / 128 * 2.0 ** 32
    lw.Wd[0, :, 0] = -(2.0 ** -10)
    lw.Wd[0, 6, 1] = 2.0 ** 14  # times h = 0; the largest weight, which leaves h unscaled
    st = D._stack(wl)
    try:
        Y = torch.zeros(T, 256, device="cuda")
        st.decode(0, wl.X.cuda(), wl.logits[0].cuda(), Y)
        D._ok(st)
        want = -float("inf") if infinite else -(181 / 128) ** 2 * 2.0 ** 117
        assert bool((Y.double() == want).all())
    finally:
        st.close()
