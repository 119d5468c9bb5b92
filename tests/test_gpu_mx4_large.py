"""The 4-bit calls at the sizes where a launch goes down many rows a block, and where
the product takes pairs of CTAs (192 rows a slot and more); tolerances as in
test_gpu_mx4."""
import numpy as np
import pytest
import torch

from tests import test_gpu_mx4 as M

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", sorted(M.TYPES))
@pytest.mark.parametrize("R,K", [(9000, 48), (3001, 520), (701, 2080)])
def test_quantise_many_rows(R, K, dtype, fmt):
    x = M.rows(R, K, dtype)
    M.check_rows(x.double().numpy(), M._es().mx4_quantize(x.cuda(), fmt, 1.0), fmt, 1.0)
    idx = torch.randint(0, R, (2 * R,), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    bad = torch.arange(0, 2 * R, 97)
    idx[bad] = -1
    got = M._es().mx4_quantize(x.cuda(), fmt, 1.0, rows=idx.cuda())
    t = x.double()[idx.clamp(min=0).long()]
    t[bad] = float("nan")
    M.check_rows(t.numpy(), got, fmt, 1.0)


@pytest.mark.parametrize("fmt", [0, 1])
def test_quantise_far_exponents(fmt):
    """Blocks near both ends of fp32's range, next to ordinary ones in a warp."""
    x = M.rows(64, 256, "f32").double().numpy()
    x[::4] *= 2.0 ** 90
    x[1::4] *= 2.0 ** -90
    x[2::8] *= 2.0 ** 100 / np.abs(x[2::8]).max()
    t = torch.from_numpy(x).float()
    for g in (1.0, 2.0 ** 20, 2.0 ** -20):
        _codes(t, fmt, g)


def _codes(t, fmt, g):
    es = M._es()
    q, s = M.quantise(t.double().numpy(), fmt, g, es.mx4_block(fmt))
    got = es.mx4_quantize(t.cuda(), fmt, g)
    np.testing.assert_array_equal(got.scales.cpu().numpy(), s)
    have = M.unpack(got.codes)
    np.testing.assert_array_equal(np.where(have == 8, 0, have), np.where(q == 8, 0, q))


@pytest.mark.parametrize("fmt", [0, 1])
def test_swiglu_far_gates(fmt):
    """Gates where exp(-g) overflows or vanishes; a NaN or infinite gate or up value
    takes its block, and no other."""
    es = M._es()
    g = torch.tensor([-150.0, -104.0, -88.5, -70.0, -30.0, -0.0, 0.0, 1e-20, 1e-3, 30.0, 90.0, 3e4])
    K = 384
    gate = g.repeat(K // 12).expand(6, K).clone()
    up = torch.ones(6, K)
    gate[1, 40], gate[2, 100], up[3, 7], gate[4, 380] = float("nan"), float("inf"), float("-inf"), float("-inf")
    x = torch.cat([gate, up], 1)
    scale = 1.0 if fmt else 16.0  # 3e4 / (6 * 16) is inside E4M3
    back = es.mx4_dequantize(es.mx4_quantize(x.cuda(), fmt, scale, swiglu=True)).cpu().double()
    b = es.mx4_block(fmt)
    h = (gate.double() / (1 + torch.exp(-gate.double())) * up).view(6, -1, b)
    bad = torch.zeros(6, K // b, dtype=torch.bool)
    bad[1, 40 // b] = bad[2, 100 // b] = bad[3, 7 // b] = True
    # g = -inf: -inf / inf is not a number
    bad[4, 380 // b] = True
    got = back.view(6, -1, b)
    assert torch.equal(torch.isnan(got).all(-1), bad) and torch.equal(torch.isnan(got).any(-1), bad)
    top = h.abs().amax(-1, keepdim=True)
    ok = ~bad
    # within half a step of the widest spacing (2 of 6) and the scale's rounding (1/16), of the block's maximum
    assert bool(((got - h).abs()[ok] <= (top * 0.25).expand_as(h)[ok]).all())


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("N,K", [(256, 256), (130, 1000), (520, 160), (333, 96)])
@pytest.mark.parametrize("offsets", [[0, 5, 400, 700], [0, 0, 257, 640], [3, 259, 600, 600], [0, 256, 512, 1024], [0, 1, 2, 900]])
def test_grouped_pairs(fmt, N, K, offsets):
    """Slots that end inside a tile of 256 rows, are empty or begin off its multiple,
    with rows before the first and after the last slot (zeros)."""
    R = offsets[-1] + 9
    for dtype in (torch.float32, torch.bfloat16):
        y = M.check_product(R, N, K, fmt, P=3, offsets=offsets, dtype=dtype)
        assert not bool(y[:offsets[0]].any()) and not bool(y[offsets[-1]:].any())
    assert M._es().mx4_error() == M._es().OK


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("R,N,K", [(192, 64, 64), (300, 200, 512), (511, 257, 1000), (1030, 72, 32)])
def test_pairs_strided_out(fmt, R, N, K):
    M.check_product(R, N, K, fmt, ld=N + 8 - N % 8)
    M.check_product(R, N, K, fmt, ld=N + 5, dtype=torch.bfloat16)
    M.check_product(R, N, K, fmt, ld=N + 5)
    M.check_product(R, N, K, fmt, spread=24)


def test_pairs_nan_scales():
    es = M._es()
    for fmt, nan in ((0, 0x7f), (1, 0xff)):
        for K in (128, 512):
            xc, xs = M.operand(400, K, fmt, 1)
            wc, ws = M.operand(300, K, fmt, 2)
            xs[3, 1] = xs[399, -1] = nan
            ws[140, 0] = ws[299, -1] = nan
            y = es.mx4_product(es.Mx4(xc.cuda(), xs.cuda(), K, fmt), es.mx4_weights(wc.cuda(), ws.cuda(), K, fmt),
                               out_dtype=torch.float32)
            nans = torch.isnan(y).cpu()
            assert bool(nans[[3, 399]].all()) and bool(nans[:, [140, 299]].all())
            nans[[3, 399]], nans[:, [140, 299]] = False, False
            assert not bool(nans.any())
