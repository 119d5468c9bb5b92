"""Chains of 4-bit calls over the same buffers, back to back in one graph: each kernel
starts while the one before it still runs, and has to see what that one wrote."""
import pytest
import torch

from tests import test_gpu_mx4 as M

pytestmark = pytest.mark.gpu


def _replay(calls):
    calls()  # first-call work
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    return g


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("R,K", [(1, 64), (1, 2048), (3, 1000), (40, 4096), (600, 512)])
def test_one_buffer_for_every_step(R, K, fmt):
    """quantise -> read back -> product of row i, for 100 different i, through one pair
    of codes and scales: every step's result is that of calls made one at a time."""
    es = M._es()
    n, N = 100, 192
    x = torch.stack([M.rows(R, K, "bf16", seed=i) * 2.0 ** (i % 7 - 3) for i in range(n)]).cuda()
    wq = es.mx4_quantize(M.rows(N, K, "bf16", seed=1000).cuda(), fmt)
    w = es.mx4_weights(wq.codes, wq.scales, K, fmt)
    q = es.mx4_quantize(x[0], fmt)
    back, y = torch.zeros(n, R, K, device="cuda"), torch.zeros(n, R, N, device="cuda")
    want_back, want_y = torch.zeros_like(back), torch.zeros_like(y)
    for i in range(n):
        es.mx4_quantize(x[i], fmt, out=q)
        torch.cuda.synchronize()
        es.mx4_dequantize(q, out=want_back[i])
        es.mx4_product(q, w, out=want_y[i])
        torch.cuda.synchronize()

    def steps():
        for i in range(n):
            es.mx4_quantize(x[i], fmt, out=q)
            es.mx4_dequantize(q, out=back[i])
            es.mx4_product(q, w, out=y[i])

    g = _replay(steps)
    for _ in range(20):
        back.zero_()
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(back, want_back)
        assert torch.equal(y, want_y)
    assert es.mx4_error() == es.OK


@pytest.mark.parametrize("fmt", [0, 1])
def test_read_back_into_the_next_source(fmt):
    """quantise -> read back into the rows that the next step quantises, scaled by the
    next step's tensor scale: 100 steps against the same ones one at a time."""
    es = M._es()
    x0 = M.rows(2, 512, "f32", seed=5).cuda()
    x, other = x0.clone(), torch.empty_like(x0)
    scales = [2.0 ** (i % 3 - 1) * (1.0 + (i % 5) / 7) for i in range(100)]
    q = es.mx4_quantize(x, fmt)

    def steps(wait):
        a, b = x, other
        for s in scales:
            es.mx4_quantize(a, fmt, s, out=q)
            wait()
            es.mx4_dequantize(q, out=b)
            wait()
            a, b = b, a

    steps(torch.cuda.synchronize)
    want = x.clone()
    x.copy_(x0)
    g = _replay(lambda: steps(lambda: None))
    for _ in range(20):
        x.copy_(x0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, want)
