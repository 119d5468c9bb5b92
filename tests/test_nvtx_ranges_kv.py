"""NVTX ranges of the cache's calls and of sampling, recorded as in test_nvtx_ranges."""
from tests.test_nvtx_ranges import _record, _tree, recorder  # noqa: F401 (fixture)


def test_ranges_of_cache_and_sampling_calls(recorder, tmp_path):  # noqa: F811
    """A call opens its range before it looks at its arguments: refused ones record it."""
    code = """
from routed_expert_ffn_topk_gb300 import estream as es
L = es.lib()
N = None
assert L.estream_kv_append(N, 0, 7, N, 0, 0, N, 0, 0, N, N, N, 0, 0, 0, N, 0, 0, 0, N, 0, 0, N, 0, 0, N) == es.ERR_INVALID_ARG
assert L.estream_kv_attend(N, 0, 5, 2, N, 0, 0, N, 1, 0, N, 1.0, 0, N, 0, 0, N, N, 0, N) == es.ERR_INVALID_ARG
assert L.estream_sample_tokens(N, 2, 0, 3, 8, N, 1.0, N, 0, N, 1.0, N, 0.0, N, N, N, N) == es.ERR_INVALID_ARG
"""
    assert _tree(_record(recorder, tmp_path, code)) == [
        ("cache append", 7, None), ("cache attend", 5, None), ("sample", 3, None)]
