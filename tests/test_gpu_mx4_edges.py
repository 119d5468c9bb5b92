"""The microscaled 4-bit calls at the ends of their argument ranges."""
import pytest
import torch

from tests import test_gpu_mx4 as M

pytestmark = pytest.mark.gpu


def test_offsets_that_count_rows_many_times():
    """2048 slots that each claim every one of 671 million rows are more row tiles
    than 32 bits hold: nothing outside the result is touched, no wait runs out, and
    the same sizes with ascending offsets give their values."""
    es = M._es()
    R, P, K = 5 << 27, 4096, 32
    x = es.Mx4(torch.full((R, 16), 0x22, dtype=torch.uint8, device="cuda"),
               torch.full((R, 1), 127, dtype=torch.uint8, device="cuda"), K, 1)
    w = es.mx4_weights(torch.full((P, 1, 16), 0x22, dtype=torch.uint8, device="cuda"),
                       torch.full((P, 1, 1), 127, dtype=torch.uint8, device="cuda"), K, 1)
    buf = torch.full((R + 128, 1), 5.0, device="cuda")
    claims = torch.zeros(P + 1, dtype=torch.int32)
    claims[1::2] = R
    even = (torch.arange(P + 1, dtype=torch.int64) * (R // P)).to(torch.int32)
    for off in (claims, even):
        es.mx4_product(x, w, offsets=off.cuda(), out=buf[64:-64])
        torch.cuda.synchronize()
        assert bool((buf[:64] == 5.0).all()) and bool((buf[-64:] == 5.0).all())
        assert es.mx4_error() == es.OK
    assert bool((buf[64:-64] == 32.0).all())  # 32 products of 1 and 1


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("fmt", [0, 1])
def test_gather_from_no_rows(fmt, swiglu):
    """Every index is out of range of a source without rows: rows of NaNs."""
    es = M._es()
    x = torch.empty(0, 128 if swiglu else 64, dtype=torch.bfloat16, device="cuda")
    idx = torch.tensor([0, -1, 5], dtype=torch.int32).cuda()
    q = es.mx4_quantize(x, fmt, rows=idx, swiglu=swiglu)
    assert q.shape == (3, 64) and bool(torch.isnan(es.mx4_dequantize(q)).all())


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("P,rows", [(65, 192), (70, 260), (130, 200)])
def test_pairs_of_many_slots(P, rows, fmt):
    """More than 64 slots of 192 rows and more: the pair form with its slots' prefix
    beside the ring."""
    g = torch.Generator().manual_seed(P)
    n = torch.randint(rows - 40, rows + 60, (P,), generator=g)
    n[3], n[P - 2] = 0, 1
    n[7] += max(0, P * rows - int(n.sum()))  # 192 rows a slot on average at least
    off = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).tolist()
    for N, K, dtype in ((256, 512, torch.bfloat16), (130, 96, torch.float32)):
        M.check_product(off[-1], N, K, fmt, P=P, offsets=off, dtype=dtype)
    assert M._es().mx4_error() == M._es().OK
