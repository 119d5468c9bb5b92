"""Limits of the microscaled 4-bit calls' sizes, without a GPU: a size past a limit is
an argument error, reported before anything touches CUDA."""
import ctypes

import pytest

from routed_expert_ffn_topk_gb300 import build as build_mod


@pytest.fixture(scope="module")
def es():
    build_mod.build()
    from routed_expert_ffn_topk_gb300 import estream
    return estream


@pytest.mark.parametrize("R", [(1 << 30) + 1, 2 ** 31 - 7296, 2 ** 31 - 1])
def test_rows_past_the_limit(es, R):
    """Row indices and their strides are 32-bit: 2^30 rows in every call."""
    L = es.lib()
    buf = (ctypes.c_char * 4096)()
    p = (ctypes.addressof(buf) + 255) & ~255
    for rows in (None, p):
        assert L.estream_mx4_quantize(p, 0, 32, R, R, 32, rows, 0, 0, 1.0, p, p, None) == es.ERR_INVALID_ARG
    assert L.estream_mx4_dequantize(p, p, 0, 1.0, R, 32, p, 2, 32, None) == es.ERR_INVALID_ARG
    assert L.estream_mx4_product(p, p, R, p, p, 1, 8, 32, 0, 1.0, None, p, 2, 8, None) == es.ERR_INVALID_ARG
