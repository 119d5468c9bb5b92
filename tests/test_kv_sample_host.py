"""Argument errors of the cache's calls and of sampling, without a GPU: status codes come back before
anything touches CUDA."""
import ctypes

import pytest
import torch

from routed_expert_ffn_topk_gb300 import build as build_mod


@pytest.fixture(scope="module")
def es():
    build_mod.build()
    from routed_expert_ffn_topk_gb300 import estream
    return estream


@pytest.fixture
def p():
    buf = (ctypes.c_char * 4096)()
    yield (ctypes.addressof(buf) + 255) & ~255


def _cache(es, p, **kw):
    d = dict(k=p, v=p, elem=es.KV_BF16, num_pages=4, page_size=16, heads=2, dim=64, k_scale=1.0, v_scale=1.0,
             k_page=2048, k_token=128, k_head=64, v_page=2048, v_token=128, v_head=64)
    d.update(kw)
    return es.KvCache(**d)


BAD_CACHES = [dict(elem=3), dict(elem=-1), dict(num_pages=-1), dict(page_size=0), dict(heads=0), dict(heads=1025), dict(dim=0),
              dict(dim=40), dict(dim=272), dict(k_scale=0.5), dict(v_scale=float("nan")), dict(elem=2, k_scale=0.0),
              dict(elem=2, v_scale=float("inf")), dict(elem=2, k_scale=2.0 ** -101), dict(k_page=2052), dict(k_token=60),
              dict(v_head=-64), dict(v_page=0), dict(k=None), dict(elem=2, k_head=72)]


def test_caches(es, p):
    L = es.lib()

    def append(c):
        return L.estream_kv_append(ctypes.byref(c), 0, 0, None, 0, 0, None, 0, 0, None, None, None, 0, 0, 0, None, 0, 0, 0,
                                   None, 0, 0, None, 0, 0, None)

    def attend(c):
        return L.estream_kv_attend(ctypes.byref(c), 0, 0, 2, None, 0, 0, None, 1, 0, None, 1.0, 0, None, 0, 0, None, None, 0, None)

    for call in (append, attend):
        assert call(_cache(es, p)) == es.OK
        assert call(_cache(es, p, num_pages=0, k=None, v=None)) == es.OK
        assert call(_cache(es, p, num_pages=1, k_page=0, v_page=0)) == es.OK  # one page: its stride is not used
        for kw in BAD_CACHES:
            assert call(_cache(es, p, **kw)) == es.ERR_INVALID_ARG, kw
    assert L.estream_kv_append(None, 0, 0, None, 0, 0, None, 0, 0, None, None, None, 0, 0, 0, None, 0, 0, 0,
                               None, 0, 0, None, 0, 0, None) == es.ERR_INVALID_ARG


def test_append_arguments(es, p):
    L, c = es.lib(), _cache(es, p)

    def call(c=c, elem=0, T=2, k=p, v=p, positions=p, rows=p, table=p, B=2, M=1, table_row=1, q=p, Hq=4, q_out=p, inv=p, rot=64):
        return L.estream_kv_append(ctypes.byref(c), elem, T, k, 128, 64, v, 128, 64, positions, rows, table, B, M, table_row,
                                   q, 256, 64, Hq, q_out, 256, 64, inv, rot, 0, None)

    for kw in (dict(elem=1), dict(elem=2), dict(T=-1), dict(T=(1 << 24) + 1), dict(k=None), dict(v=p + 1), dict(positions=None),
               dict(positions=p + 2), dict(rows=p + 1), dict(table=None), dict(B=-1), dict(M=-1), dict(table_row=-1),
               dict(q=None), dict(q_out=None), dict(q=p + 1), dict(Hq=-1), dict(Hq=1025), dict(inv=None), dict(rot=-2),
               dict(rot=3), dict(rot=66)):
        assert call(**kw) == es.ERR_INVALID_ARG, kw
    assert call(T=0, k=None) == es.OK


def test_attend_arguments(es, p):
    L, c = es.lib(), _cache(es, p)

    def call(c=c, elem=0, B=2, Hq=4, q=p, table=p, M=1, table_row=1, lens=p, scale=1.0, window=0, out=p, lse=p, ws=p, n=1 << 30):
        return L.estream_kv_attend(ctypes.byref(c), elem, B, Hq, q, 256, 64, table, M, table_row, lens, scale, window,
                                   out, 256, 64, lse, ws, n, None)

    for kw in (dict(elem=1), dict(elem=2), dict(B=-1), dict(Hq=0), dict(Hq=3), dict(B=1 << 20, Hq=32), dict(q=None), dict(q=p + 1),
               dict(table=None), dict(table=p + 2), dict(M=-1), dict(M=1 << 28), dict(table_row=-1), dict(lens=None),
               dict(lens=p + 1), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(out=None),
               dict(lse=p + 2)):
        assert call(**kw) == es.ERR_INVALID_ARG, kw
    assert call(B=0, q=None) == es.OK
    assert L.estream_kv_attend_workspace_bytes(ctypes.byref(c), 0, 4, 1, 0) == 0
    assert L.estream_kv_attend_workspace_bytes(ctypes.byref(c), 2, 3, 1, 0) == 0


def test_sample_arguments(es, p):
    L = es.lib()

    def call(l=p, elem=2, ld=100, B=2, V=100, u=p, t=None, k=None, tp=None, m=None, ids=p, prob=p):
        return L.estream_sample_tokens(l, elem, ld, B, V, u, 1.0, t, 0, k, 1.0, tp, 0.0, m, ids, prob, None)

    for kw in (dict(l=None), dict(l=p + 2), dict(elem=3), dict(elem=-1), dict(ld=-1), dict(B=-1), dict(B=(1 << 20) + 1), dict(V=0),
               dict(V=es.SAMPLE_MAX_V + 1, ld=1 << 20), dict(u=None), dict(u=p + 1), dict(t=p + 2), dict(k=p + 1), dict(tp=p + 1),
               dict(m=p + 3), dict(ids=None), dict(ids=p + 2), dict(prob=p + 1)):
        assert call(**kw) == es.ERR_INVALID_ARG, kw
    assert call(B=0, l=None) == es.OK


def test_tensors_on_the_cpu_are_refused(es):
    k = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        es.PagedKV(k, k)
    with pytest.raises(ValueError):
        es.sample_tokens(torch.zeros(2, 10), torch.zeros(2))


def test_division_by_constants(tmp_path):
    """The kernels' division by a page's size, over the divisors' edges and numbers next to their multiples."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "div.cu"
    src.write_text("""
#include <cstdio>
#include "estream_internal.h"
int main() {
    for (uint64_t e = 0; e <= 30; ++e)
        for (int64_t off = -2; off <= 2; ++off) {
            const int64_t d = (int64_t(1) << e) + off;
            if (d < 1 || d > (int64_t(1) << 30)) continue;
            const es::FastDiv f(static_cast<uint32_t>(d));
            for (uint64_t q = 0; q < 2000; ++q)
                for (int64_t k = -1; k <= 1; ++k) {
                    const int64_t top = 0x7fffffffll / d, m = q < 1000 ? int64_t(q) : top - (int64_t(q) - 1000);
                    const int64_t n = m * d + k;
                    if (n < 0 || n > 0x7fffffffll) continue;
                    if (f.div(static_cast<uint32_t>(n)) != n / d) return printf("%lld / %lld\\n", (long long)n, (long long)d), 1;
                }
        }
    return 0;
}
""")
    exe = tmp_path / "div"
    pkg = os.path.join(root, "routed_expert_ffn_topk_gb300", "csrc")
    subprocess.run([build_mod._nvcc(), "-std=c++17", "-I" + pkg, "-I" + os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    subprocess.run([str(exe)], check=True)
