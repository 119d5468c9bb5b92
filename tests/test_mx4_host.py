"""Sizes and argument errors of the microscaled 4-bit and few-token calls, without
a GPU: status codes come back before anything touches CUDA."""
import ctypes

import pytest

from routed_expert_ffn_topk_gb300 import build as build_mod


@pytest.fixture(scope="module")
def es():
    build_mod.build()
    from routed_expert_ffn_topk_gb300 import estream
    return estream


def test_sizes(es):
    L = es.lib()
    assert [es.mx4_padded(k) for k in (1, 32, 33, 2048)] == [32, 32, 64, 2048]
    assert L.estream_mx4_code_bytes(3, 33) == 3 * 32
    assert L.estream_mx4_scale_bytes(3, 33, es.FP4_E4M3X16) == 3 * 4
    assert L.estream_mx4_scale_bytes(3, 33, es.FP4_E8M0X32) == 3 * 2
    assert L.estream_mx4_weight_scale_bytes(2, 129, 65) == 2 * 2 * 2 * 512
    assert L.estream_mx4_code_bytes(-1, 33) == 0 == L.estream_mx4_code_bytes(1, 0)
    assert L.estream_mx4_scale_bytes(1, 32, 2) == 0 == L.estream_mx4_weight_scale_bytes(0, 1, 1)
    # past 32 bits
    assert L.estream_mx4_code_bytes(1 << 20, 1 << 14) == 1 << 33


def test_tensor_scale(es):
    s = es.mx4_tensor_scale(100.0, es.FP4_E4M3X16)
    assert 224 < 100.0 / (6 * s) <= 448 and s == 2.0 ** round(__import__("math").log2(s))
    assert es.mx4_tensor_scale(100.0, es.FP4_E8M0X32) == 1.0
    for a in (0.0, float("nan"), float("inf")):
        assert es.mx4_tensor_scale(a, es.FP4_E4M3X16) == 1.0
    with pytest.raises(ValueError):
        es.mx4_block(2)


def test_argument_errors(es):
    L = es.lib()
    buf = (ctypes.c_char * 4096)()
    p = (ctypes.addressof(buf) + 255) & ~255

    def quant(elem=0, ld=64, n=4, R=4, K=64, swiglu=0, fmt=0, scale=1.0, x=p, codes=p, scales=p):
        return L.estream_mx4_quantize(x, elem, ld, n, R, K, None, swiglu, fmt, scale, codes, scales, None)

    for kw in (dict(elem=3), dict(ld=63), dict(n=3), dict(R=-1), dict(K=0), dict(swiglu=1), dict(fmt=2), dict(scale=0.0),
               dict(scale=float("nan")), dict(x=None), dict(x=p + 1), dict(codes=p + 8), dict(codes=None),
               dict(scales=None), dict(K=(1 << 24) + 1, ld=1 << 25)):
        assert quant(**kw) == es.ERR_INVALID_ARG, kw
    assert quant(R=0, x=None) == es.OK

    def prod(R=4, P=1, N=8, K=64, fmt=0, scale=1.0, off=None, elem=2, ld=8, xc=p, xs=p, wc=p, wt=p, out=p):
        return L.estream_mx4_product(xc, xs, R, wc, wt, P, N, K, fmt, scale, off, out, elem, ld, None)

    for kw in (dict(R=-1), dict(P=0), dict(P=2), dict(P=5000, off=p), dict(N=0), dict(K=0), dict(fmt=9), dict(scale=-1.0),
               dict(elem=1), dict(ld=7), dict(xc=None), dict(xc=p + 2), dict(xs=None), dict(wc=p + 4), dict(wt=p + 16),
               dict(out=p + 2), dict(out=None), dict(off=p + 1)):
        assert prod(**kw) == es.ERR_INVALID_ARG, kw
    assert prod(R=0, xc=None) == es.OK
    assert L.estream_mx4_dequantize(p, p, 0, 1.0, 4, 64, p, 2, 63, None) == es.ERR_INVALID_ARG
    assert L.estream_mx4_weight_scales(p, 1, 8, 64, 0, p + 16, None) == es.ERR_INVALID_ARG


def test_few_token_calls_need_a_context(es):
    L = es.lib()
    assert L.estream_moe_layer_decode(None, 0, None, None, 1, 1, 0, None, None, None) == es.ERR_NOT_BOUND
    assert L.estream_moe_layer_decode_from_x(None, 0, None, None, 1, 1, 0, None, None, None, None) == es.ERR_NOT_BOUND
