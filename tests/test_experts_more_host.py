"""Arguments of the norm's and the experts' entry points at their edges, without a
GPU: what holds nothing may have any address."""
import ctypes

import pytest
import torch

from test_experts_host import A, INVALID, fq, struct  # noqa: F401

PASSED = (0, 3, 6)   # done, or stopped for want of a device behind every check


def operand(fq, **k):
    return ctypes.byref(struct(fq, **dict(dict(rows=0), **k)))


def weights(fq, **k):
    return ctypes.byref(struct(fq, **dict(dict(off=None, rows=4 * 32), **k)))


@pytest.mark.parametrize("given", [dict(q=None), dict(q=None, qt=None), dict(qs=None), dict(qts=None), {},
                                   dict(q=None, qs=None, qt=None, qts=None)])
def test_operands_of_no_rows_are_served(fq, given):
    lib = fq.lib()
    for index, T, x in ((None, 0, None), (None, 100, A), (A, 100, A)):
        assert lib.fp8_quantize_experts(x, fq.DT_BF16, T, 64, index, operand(fq, **given), None) in PASSED
    # N = 32, K = 64; the result of no rows is null too
    for y in (None, A):
        assert lib.fp8_experts_fprop(operand(fq, **given), weights(fq), y, fq.DT_BF16, None) in PASSED
        assert lib.fp8_experts_dgrad(operand(fq, cols=32, **given), weights(fq), y, fq.DT_F32, None) in PASSED


@pytest.mark.skipif(torch.cuda.is_available(), reason="would clear a result at a placeholder pointer")
def test_gradient_of_no_rows_is_served(fq):
    for given in (dict(q=None), dict(q=None, qs=None), {}):
        assert fq.lib().fp8_experts_wgrad(operand(fq, cols=32, **given), operand(fq, **given), A, fq.DT_BF16,
                                          None) in PASSED
    assert fq.lib().fp8_experts_wgrad(operand(fq, cols=32), operand(fq), None, fq.DT_BF16, None) == INVALID


def test_operands_of_no_columns_are_served(fq):
    none = dict(rows=256, cols=0, q=None, qs=None, qt=None, qts=None)
    for k in ({}, dict(q=0x10000), dict(qts=0x40000)):
        assert fq.lib().fp8_quantize_experts(None, fq.DT_BF16, 256, 0, None, operand(fq, **dict(none, **k)), None) in PASSED


def test_half_a_pair_is_still_refused(fq):
    for k in ("q", "qs", "qt", "qts"):
        assert fq.lib().fp8_quantize_experts(A, fq.DT_BF16, 256, 64, None, operand(fq, rows=256, **{k: None}),
                                             None) == INVALID
    assert fq.lib().fp8_quantize_experts(A, fq.DT_BF16, 255, 64, None, operand(fq, rows=256), None) == INVALID


@pytest.mark.parametrize("T,C", [(5, 0), (0, 64), (0, 0)])
def test_norm_of_nothing_is_served(fq, T, C):
    eps = ctypes.byref(ctypes.c_float(1e-6))
    for scaling in (fq.SCALE_ROW, fq.SCALE_TILE_1x128):
        for q, s in ((None, A), (A, None), (None, None)):
            for r, h in ((None, None), (None, A), (A, None)):
                assert fq.lib().fp8_rmsnorm(None, C, r, C, fq.DT_BF16, None, fq.DT_F32, eps, T, C, h, C, None, C,
                                            scaling, q, s, A, None) in PASSED
    assert fq.lib().fp8_rmsnorm(None, C, None, C, fq.DT_BF16, None, fq.DT_F32, eps, T, C, None, C, None, C,
                                fq.SCALE_TENSOR, A, A, A, None) == INVALID


def test_offsets_are_the_same_by_their_memory(fq):
    a = torch.tensor([0, 3, 5, 9, 9, 12], dtype=torch.int32)
    assert fq._same_offsets(a, a) and fq._same_offsets(None, None)
    assert fq._same_offsets(a, a[:]) and fq._same_offsets(a.view(-1), a)
    for other in (None, a.clone(), a[:5], a[1:], a.view(torch.float32), a[::1].view(2, 3), a[::2]):
        assert not fq._same_offsets(a, other) and not fq._same_offsets(other, a)
    assert not fq._same_offsets(a[::2], a[:3])


def test_an_operand_keeps_what_it_was_made_of(fq):
    """The calls use addresses found once: an attribute that could be set would be
    read by none of them."""
    op = fq.ExpertsOperand(64, 32, 2, fq.E5M2)
    assert (op.rows, op.cols, op.groups, op.fmt) == (64, 32, 2, fq.E5M2)
    assert op.tensors() == (None,) * 5 and op.offsets is None and op.q is None and op.qt_scales is None
    for name in ("rows", "cols", "groups", "fmt", "offsets", "q", "q_scales", "q_t", "qt_scales"):
        with pytest.raises(AttributeError):
            setattr(op, name, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(AttributeError):
        op.another = 1
