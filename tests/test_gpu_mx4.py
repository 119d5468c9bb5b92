"""Microscaled 4-bit quantisation, its inverse and the product, against plain
implementations in fp64.

Codes and scales are exact (the format's steps are reproducible, and with a
power-of-two tensor scale they are those of exact arithmetic). The product's
tolerance: operands are exact, sums are in fp32 over blocks, so
|error| <= (K / 16 + 16) 2^-23 sum |x w|, plus half a unit of the output type."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _es():
    from routed_expert_ffn_topk_gb300 import estream as es
    return es


def e4m3_values():
    """Value of each of the 127 finite non-negative E4M3 codes."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def nearest_even(table, x):
    """Index of the entry of an ascending table nearest to each x >= 0 (past the
    end: the last), ties to the even index."""
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = x - table[lo], table[hi] - x
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantise(x, fmt, g, block):
    """Codes [R, Kp], scales [R, Kp / block] of fp64 rows, from the format's
    definition (g a power of two: every step is exact in fp64)."""
    R, K = x.shape
    x = np.concatenate([x, np.zeros((R, -K % 32))], axis=1).reshape(R, -1, block)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    top = np.abs(x).max(-1)
    if fmt == 0:
        s = nearest_even(e4m3_values(), top / (6.0 * g))
        d = e4m3_values()[s] * g
        s = np.where(bad, 0x7f, s)
    else:
        e = np.where(top > 0, np.frexp(np.where(top > 0, top / g, 1.0))[1] - 1 - 2, -126)
        e = np.maximum(e, -126)
        s, d = np.where(bad, 0xff, e + 127), 2.0 ** e * g
    safe = np.where(d > 0, d, 1.0)
    q = nearest_even(E2M1, np.minimum(np.abs(x) / safe[..., None], 6.0))
    q = np.where((d > 0)[..., None], q | np.where(np.signbit(x), 8, 0), 0)
    q = np.where(bad[..., None], 0, q)
    return q.reshape(R, -1), s


def unpack(codes):
    c = codes.cpu().numpy()
    return np.stack([c & 15, c >> 4], -1).reshape(c.shape[0], -1)


def values(q, s, fmt, g, block):
    d = np.where(s == 0xff, np.nan, 2.0 ** (s.astype(np.float64) - 127)) if fmt else \
        np.where(s == 0x7f, np.nan, e4m3_values()[np.minimum(s, 126)])
    v = np.concatenate([E2M1, -E2M1])[q]
    return (v.reshape(q.shape[0], -1, block) * (d * g)[..., None]).reshape(q.shape[0], -1)


def rows(R, K, dtype, seed=1, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, K, generator=g) * torch.exp(torch.randn(R, K, generator=g) * spread / 3)
    return x.to(TYPES[dtype])


def check_rows(x64, got, fmt, g):
    es = _es()
    block = es.mx4_block(fmt)
    q, s = quantise(x64, fmt, g, block)
    np.testing.assert_array_equal(got.scales.cpu().numpy(), s)
    have = unpack(got.codes)
    # the sign of a zero carries no value
    np.testing.assert_array_equal(np.where(have == 8, 0, have), np.where(q == 8, 0, q))
    for name, dt in TYPES.items():
        back = es.mx4_dequantize(got, dt).double().cpu().numpy()
        want = values(q, s, fmt, g, block)[:, :x64.shape[1]]
        if name == "f16":
            want = torch.from_numpy(want).half().double().numpy()
        np.testing.assert_array_equal(back, want)


@pytest.mark.parametrize("fmt,g", [(0, 1.0), (0, 2.0 ** -6), (1, 1.0), (1, 4.0)])
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("R,K", [(1, 1), (1, 2048), (3, 31), (2, 32), (5, 33), (7, 1000), (64, 16), (1021, 48), (33, 4096)])
def test_quantise(R, K, dtype, fmt, g):
    x = rows(R, K, dtype)
    check_rows(x.double().numpy(), _es().mx4_quantize(x.cuda(), fmt, g), fmt, g)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_ties_zeros_and_extremes(fmt, dtype):
    """Values on every rounding boundary, blocks of zeros, of the smallest and
    largest magnitudes, and blocks with a NaN or an infinity."""
    mid = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1, 1.5, 2, 3, 4, -0.25, -5.0])
    x = np.zeros((12, 64))
    for r in range(6):
        x[r, :16] = mid * 2.0 ** (r - 3)
        x[r, 16:32] = -mid * 2.0 ** (r - 3) * 1.5
        x[r, 32:48] = mid[::-1] * 1.125
    x[7, :] = 2.0 ** -14
    x[8, 3], x[8, 40] = np.nan, 1.0
    x[9, 5], x[9, 20] = np.inf, -2.0
    x[10, 63] = -np.inf
    x[11, :] = 65504.0 if dtype == "f16" else 2.0 ** 100
    t = torch.from_numpy(x).to(TYPES[dtype])
    check_rows(t.double().numpy(), _es().mx4_quantize(t.cuda(), fmt, 1.0), fmt, 1.0)
    if dtype != "f16":
        t = torch.full((2, 32), 2.0 ** -126).to(TYPES[dtype])
        t[1] = float(torch.finfo(TYPES[dtype]).max)
        check_rows(t.double().numpy(), _es().mx4_quantize(t.cuda(), fmt, 1.0), fmt, 1.0)


@pytest.mark.parametrize("fmt", [0, 1])
def test_any_tensor_scale(fmt):
    """A tensor scale that is no power of two: each step is one fp32 operation."""
    es = _es()
    x = rows(50, 320, "f32")
    g = np.float32(0.0317)
    got = es.mx4_quantize(x.cuda(), fmt, float(g))
    b = es.mx4_block(fmt)
    xs = x.numpy().reshape(50, -1, b)
    top = np.abs(xs).max(-1)
    if fmt == 0:
        s = nearest_even(e4m3_values(), (top / (np.float32(6) * g)).astype(np.float64))
        d = e4m3_values()[s].astype(np.float32) * g
    else:
        s = np.frexp(top / g)[1] - 3 + 127
        d = (2.0 ** (s - 127)).astype(np.float32) * g
    q = nearest_even(E2M1, np.minimum(np.abs(xs / d[..., None]).astype(np.float64), 6.0)) | (np.signbit(xs) * 8)
    np.testing.assert_array_equal(got.scales.cpu().numpy(), s)
    np.testing.assert_array_equal(unpack(got.codes), q.reshape(50, -1))
    back = es.mx4_dequantize(got).cpu().numpy().reshape(xs.shape)
    v = np.concatenate([E2M1, -E2M1]).astype(np.float32)[q]
    np.testing.assert_array_equal(back, v * d[..., None])


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_gather_and_strides(fmt, dtype):
    """Rows by index (with repeats), source rows further apart than they are
    long, a base off a 16-byte boundary; an index out of range reads as NaN."""
    es = _es()
    for K, ld, off in ((160, 160, 0), (160, 192, 0), (96, 97, 0), (64, 80, 3), (50, 64, 8)):
        big = rows(40, ld, dtype)
        x = big[:, off:off + K] if off + K <= ld else big[:, :K]
        idx = torch.randint(0, 40, (100,), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
        dev = big.cuda()
        view = dev[:, off:off + K] if off + K <= ld else dev[:, :K]
        check_rows(x[idx.long()].double().numpy(), es.mx4_quantize(view, fmt, 1.0, rows=idx.cuda()), fmt, 1.0)
        check_rows(x.double().numpy(), es.mx4_quantize(view, fmt, 1.0), fmt, 1.0)
        bad = torch.tensor([3, -1, 40, 2 ** 31 - 1, 0], dtype=torch.int32)
        back = es.mx4_dequantize(es.mx4_quantize(view, fmt, 1.0, rows=bad.cuda())).cpu()
        assert bool(torch.isnan(back[1:4]).all()) and bool(torch.isfinite(back[[0, 4]]).all())


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("K", [1, 17, 64, 352])
def test_swiglu(fmt, K):
    """SiLU(gate) * up in fp32, each step rounded once; the exponential is CUDA's,
    at most 2 ulp off, so codes may differ where the value meets a boundary to
    that precision and nowhere else."""
    es = _es()
    gu = rows(60, 2 * K, "bf16", spread=1.0)
    got = es.mx4_dequantize(es.mx4_quantize(gu.cuda(), fmt, 1.0 if fmt else 2.0 ** -4, swiglu=True)).cpu().numpy()
    g, u = gu[:, :K].double().numpy(), gu[:, K:].double().numpy()
    h = g / (1 + np.exp(-g)) * u
    block = es.mx4_block(fmt)
    near = []
    for f in (1 - 2.0 ** -20, 1.0, 1 + 2.0 ** -20):
        q, s = quantise(h * f, fmt, 1.0 if fmt else 2.0 ** -4, block)
        near.append(values(q, s, fmt, 1.0 if fmt else 2.0 ** -4, block)[:, :K])
    ok = (got == near[0]) | (got == near[1]) | (got == near[2])
    assert ok.all()
    assert (got == near[1]).mean() > 0.999


def test_past_32_bits():
    """More than 2^31 values: the last rows of a large matrix."""
    es = _es()
    R, K = 70000, 32768
    x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    tail = rows(64, K, "bf16")
    x[-64:] = tail.cuda()
    q = es.mx4_quantize(x, 0, 1.0)
    del x
    part = es.Mx4(q.codes[-64:].contiguous(), q.scales[-64:].contiguous(), K, 0, 1.0)
    check_rows(tail.double().numpy(), part, 0, 1.0)
    out = es.mx4_dequantize(q, torch.bfloat16)
    want = es.mx4_dequantize(part, torch.bfloat16)
    assert torch.equal(out[-64:], want) and not bool(out[:64].any())


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------

def operand(R, K, fmt, seed, spread=4):
    """Random codes and scales of rows of K (codes past K zero)."""
    es = _es()
    g = torch.Generator().manual_seed(seed)
    Kp, b = es.mx4_padded(K), es.mx4_block(fmt)
    c = torch.randint(0, 256, (R, Kp // 2), generator=g, dtype=torch.uint8)
    c[:, (K + 1) // 2:] = 0
    if K % 2:
        c[:, K // 2] &= 15
    lo = max(0, 0x38 - 8 * (spread // 2)) if fmt == 0 else 127 - spread // 2
    hi = min(0x7f, 0x38 + 8 * (spread // 2)) if fmt == 0 else 127 + spread // 2
    s = torch.randint(lo, hi, (R, Kp // b), generator=g, dtype=torch.uint8)
    return c, s


def wide(c, s, fmt):
    return torch.from_numpy(values(unpack(c), s.numpy(), fmt, 1.0, 32 if fmt else 16)).cuda()


def check_product(R, N, K, fmt, P=1, offsets=None, dtype=torch.float32, scales=(1.0, 1.0), spread=4, ld=None):
    es = _es()
    xc, xs = operand(R, K, fmt, 1, spread)
    wc, ws = operand(P * N, K, fmt, 2, spread)
    x = es.Mx4(xc.cuda(), xs.cuda(), K, fmt, scales[0])
    w = es.mx4_weights(wc.view(P, N, -1).cuda(), ws.view(P, N, -1).cuda(), K, fmt, scales[1])
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32).cuda()
    out = None
    if ld:
        buf = torch.full((R, ld), 99.0, dtype=dtype, device="cuda")
        out = buf[:, :N]
    y = es.mx4_product(x, w, offsets=off, out=out, out_dtype=dtype)
    assert torch.equal(y, es.mx4_product(x, w, offsets=off, out_dtype=dtype)), "not reproducible"
    if ld:
        assert bool((buf[:, N:] == 99.0).all())
    X, Wt = wide(xc, xs, fmt) * scales[0], (wide(wc, ws, fmt) * scales[1]).view(P, N, -1)
    want, mag = torch.zeros(R, N, dtype=torch.float64, device="cuda"), torch.zeros(R, N, dtype=torch.float64, device="cuda")
    bounds = [0, R] if offsets is None else offsets
    for p in range(P):
        lo, hi = bounds[p], bounds[p + 1]
        if hi > lo:
            want[lo:hi] = X[lo:hi] @ Wt[p].t()
            mag[lo:hi] = X[lo:hi].abs() @ Wt[p].abs().t()
    tol = (K / 16 + 16) * 2.0 ** -23 * mag
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), f"worst {float((err - tol).max()):.3e}"
    return y


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("R,N,K", [
    (1, 1, 1), (1, 128, 64), (1, 4096, 2048), (2, 100, 96), (3, 129, 1000), (7, 255, 33), (8, 256, 256),
    (16, 384, 512), (17, 640, 288), (31, 77, 800), (33, 130, 2016), (64, 256, 4096), (65, 512, 1408), (128, 128, 128),
    (129, 1000, 640), (200, 333, 777), (256, 256, 256), (257, 513, 1536), (500, 96, 14336), (1000, 2048, 512)])
def test_product(R, N, K, fmt):
    check_product(R, N, K, fmt)
    check_product(R, N, K, fmt, dtype=torch.bfloat16, scales=(2.0 ** -3, 0.25))


@pytest.mark.parametrize("fmt", [0, 1])
def test_product_wide_scales_and_strided_out(fmt):
    check_product(70, 200, 512, fmt, spread=24)
    check_product(70, 200, 512, fmt, ld=208)
    check_product(70, 201, 512, fmt, ld=233, dtype=torch.bfloat16)
    check_product(1, 201, 512, fmt, ld=233, dtype=torch.bfloat16)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("N,K", [(256, 256), (130, 1000)])
@pytest.mark.parametrize("offsets", [
    [0, 5, 5, 12, 12], [0, 0, 0, 1, 1], [3, 7, 300, 301, 555], [0, 128, 256, 384, 512], [0, 129, 130, 400, 700],
    [0, 0, 0, 0, 0], [0, 1, 2, 3, 4]])
def test_grouped(fmt, N, K, offsets):
    """Slots of every size, empty ones, tiles that start off a tile's multiple, and
    rows before the first and after the last slot (zeros)."""
    R = max(offsets[-1] + 9, 20)
    for dtype in (torch.float32, torch.bfloat16):
        y = check_product(R, N, K, fmt, P=4, offsets=offsets, dtype=dtype)
        assert not bool(y[:offsets[0]].any()) and not bool(y[offsets[-1]:].any())


def test_grouped_many_slots():
    g = torch.Generator().manual_seed(4)
    n = torch.randint(0, 70, (300,), generator=g)
    n[5:20] = 0
    off = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).tolist()
    check_product(off[-1], 200, 160, 0, P=300, offsets=off)
    n = (torch.rand(300, generator=g) < 0.1).long()
    off = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).tolist()
    check_product(off[-1], 200, 160, 1, P=300, offsets=off)


def test_bad_offsets_stay_inside():
    """Offsets that descend or leave [0, R] are clamped: nothing outside is touched."""
    es = _es()
    xc, xs = operand(40, 64, 0, 1)
    wc, ws = operand(3 * 64, 64, 0, 2)
    x = es.Mx4(xc.cuda(), xs.cuda(), 64, 0)
    w = es.mx4_weights(wc.view(3, 64, -1).cuda(), ws.view(3, 64, -1).cuda(), 64, 0)
    for off in ([-5, 10, 2 ** 31 - 1, 50], [30, 10, 20, 5], [50, 60, 70, 80]):
        buf = torch.full((60, 64), 5.0, device="cuda")
        es.mx4_product(x, w, offsets=torch.tensor(off, dtype=torch.int32).cuda(), out=buf[:40])
        torch.cuda.synchronize()
        assert bool((buf[40:] == 5.0).all())


def test_nan_scales():
    """A NaN scale reaches its row (x) or column (w) and nothing else."""
    es = _es()
    for fmt, nan in ((0, 0x7f), (1, 0xff)):
        xc, xs = operand(20, 128, fmt, 1)
        wc, ws = operand(150, 128, fmt, 2)
        xs[3, 1] = nan
        ws[140, 0] = nan
        y = es.mx4_product(es.Mx4(xc.cuda(), xs.cuda(), 128, fmt), es.mx4_weights(wc.cuda(), ws.cuda(), 128, fmt),
                           out_dtype=torch.float32)
        nans = torch.isnan(y).cpu()
        assert bool(nans[3].all()) and bool(nans[:, 140].all())
        nans[3], nans[:, 140] = False, False
        assert not bool(nans.any())


def test_graph_and_stream():
    es = _es()
    x = rows(9, 256, "bf16").cuda()
    wq = es.mx4_quantize(rows(200, 256, "bf16", seed=3).cuda(), 0, 1.0)
    w = es.mx4_weights(wq.codes, wq.scales, 256, 0)

    def step(t, stream=None):
        return es.mx4_product(es.mx4_quantize(t, 0, 0.5, stream=stream), w, stream=stream)

    want = [step(x), step(x * 2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(x)
    side.synchronize()
    assert torch.equal(got, want[0])
    buf = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = step(buf)
    for k in (1, 0):
        buf.copy_(x * (1 + k))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k])


def test_refusals():
    es = _es()
    x = rows(4, 64, "bf16").cuda()
    q = es.mx4_quantize(x, 0)
    w = es.mx4_weights(q.codes, q.scales, 64, 0)
    bad = [
        lambda: es.mx4_quantize(x.double(), 0), lambda: es.mx4_quantize(x, 2), lambda: es.mx4_quantize(x.t(), 0),
        lambda: es.mx4_quantize(x, 0, rows=torch.zeros(3, device="cuda")),
        lambda: es.mx4_quantize(x[:, :63], 0, swiglu=True), lambda: es.mx4_quantize(x[0], 0),
        lambda: es.mx4_quantize(x, 1, out=q), lambda: es.mx4_quantize(x[:3], 0, out=q),
        lambda: es.mx4_quantize(x.cpu(), 0), lambda: es.mx4_dequantize(q, torch.float64),
        lambda: es.mx4_dequantize(q, out=torch.empty(4, 65, device="cuda")),
        lambda: es.Mx4(q.codes, q.scales, 63 + 32, 0), lambda: es.Mx4(q.codes, q.scales, 64, 1),
        lambda: es.Mx4(q.codes.cpu(), q.scales.cpu(), 64, 0),
        lambda: es.mx4_weights(q.codes, q.scales[:3], 64, 0), lambda: es.mx4_weights(q.codes, q.scales, 0, 0),
        lambda: es.mx4_product(es.mx4_quantize(x, 1), w), lambda: es.mx4_product(es.mx4_quantize(x[:, :32], 0), w),
        lambda: es.mx4_product(q, w, out_dtype=torch.float16),
        lambda: es.mx4_product(q, w, out=torch.empty(4, 5, device="cuda")),
        lambda: es.mx4_product(q, w, offsets=torch.zeros(1, dtype=torch.int32, device="cuda")),
        lambda: es.mx4_product(q, es.mx4_weights(q.codes.view(2, 2, -1), q.scales.view(2, 2, -1), 64, 0)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(f"call {i} was not refused")
    for f in (lambda: es.mx4_quantize(x, 0, 0.0), lambda: es.mx4_quantize(x, 0, float("nan")),
              lambda: es.mx4_quantize(x, 0, float("inf")), lambda: es.mx4_quantize(x, 0, -1.0)):
        with pytest.raises(es.EStreamError) as e:
            f()
        assert e.value.status == es.ERR_INVALID_ARG
    empty = es.mx4_quantize(x[:0], 0)
    assert empty.shape == (0, 64)
    assert es.mx4_product(empty, w).shape == (0, 4)
    assert es.mx4_dequantize(empty).shape == (0, 64)
