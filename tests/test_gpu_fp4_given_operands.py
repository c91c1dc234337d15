"""fp4_quantize into operands of the caller's: each orientation asked for is
written with its scale, one that is not asked for stays as it is."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import scaled_quantize_fp8_warp_gb300 as fq
    yield fq
    assert fq.device_status() == fq.OK


def normal(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).bfloat16().cuda()


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("rows,cols", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("give_q,give_t", [(True, False), (False, True), (True, True)])
def test_only_what_is_asked_for_is_written(fq, kind, rows, cols, give_q, give_t):
    old, x = normal((64, 96), 1), normal((64, 96), 2, 50.0)
    # two operands of an earlier matrix: with one tensor scale if one call is to write both
    q, q_t = fq.fp4_quantize(old, kind, cols=True)
    if not (rows and cols):
        q_t = fq.fp4_quantize(old, kind, rows=False, cols=True)[1]
    before = fq.fp4_dequantize(q), fq.fp4_dequantize(q_t)
    got = fq.fp4_quantize(x, kind, rows=rows, cols=cols, q=q if give_q else None, q_t=q_t if give_t else None)
    want = fq.fp4_quantize(x, kind, cols=True)
    for asked, given, mine, op, fresh, was in ((rows, give_q, q, got[0], want[0], before[0]),
                                              (cols, give_t, q_t, got[1], want[1], before[1])):
        assert (op is not None) == asked
        if asked:
            assert torch.equal(fq.fp4_dequantize(op), fq.fp4_dequantize(fresh))
            assert torch.equal(op.data, fresh.data) and torch.equal(op.scales, fresh.scales)
            assert (op is mine) == given
        elif not (rows and cols):
            assert torch.equal(fq.fp4_dequantize(mine), was)
