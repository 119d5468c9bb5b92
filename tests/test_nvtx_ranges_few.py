"""NVTX ranges of the few-token and 4-bit calls, recorded as in test_nvtx_ranges."""
import pytest

from tests.test_nvtx_ranges import _record, _tree, recorder  # noqa: F401 (fixture)


def test_ranges_of_4bit_calls(recorder, tmp_path):  # noqa: F811
    """A call opens its range before it looks at its arguments: refused ones record it."""
    code = """
from routed_expert_ffn_topk_gb300 import estream as es
L = es.lib()
assert L.estream_mx4_quantize(None, 0, 64, 3, 3, 64, None, 0, 0, 1.0, None, None, None) == es.ERR_INVALID_ARG
assert L.estream_mx4_dequantize(None, None, 0, 1.0, 4, 64, None, 2, 64, None) == es.ERR_INVALID_ARG
assert L.estream_mx4_weight_scales(None, 2, 8, 64, 0, None, None) == es.ERR_INVALID_ARG
assert L.estream_mx4_product(None, None, 5, None, None, 1, 8, 64, 0, 1.0, None, None, 2, 8, None) == es.ERR_INVALID_ARG
"""
    assert _tree(_record(recorder, tmp_path, code)) == [
        ("4-bit quantise", 3, None), ("4-bit dequantise", 4, None), ("4-bit weight scales", 16, None),
        ("4-bit product", 5, None)]


@pytest.mark.gpu
def test_ranges_of_a_few_token_call(recorder, tmp_path):  # noqa: F811
    code = """
import torch
from routed_expert_ffn_topk_gb300 import estream as es, workloads as W
from routed_expert_ffn_topk_gb300.layer import BoundLayerStack
cfg = W.scaled(W.CONFIGS["c2"], T=3, H=256, E=8, k=2, F=128)
wl = W.make_workload(cfg)
st = BoundLayerStack(wl, mode="resident")
Y = torch.zeros(cfg.T, cfg.H, device="cuda")
st.decode(0, wl.X.cuda(), wl.logits[0].cuda(), Y)
torch.cuda.synchronize()
assert es.get_device_error(st.ctx) == es.OK
st.close()
"""
    ranges = [r for r in _tree(_record(recorder, tmp_path, code)) if r[0] in ("layer", "routed experts")]
    assert ranges == [("layer", 0, None), ("routed experts", 0, "layer")]
