"""Sizes past the 32-bit row coordinates of the 4-bit products' kernels are
refused before any device work, by every entry point that runs one."""
import ctypes

import pytest

P = ctypes.c_void_p
A = P(0x10000)
INVALID = 1
PAST = [1 << 31, 2_200_000_000, (1 << 31) - 1, (1 << 33) + 128]   # the next tile's rows, or more, pass INT32_MAX


@pytest.fixture(scope="module")
def fq():
    from scaled_quantize_fp8_warp_gb300 import build_lib
    import scaled_quantize_fp8_warp_gb300 as fq
    build_lib.build()
    fq.load_library()
    return fq


def operand(fq, kind):
    return ctypes.byref(fq._Fp4Struct(0x10000, 0x20000, 0x30000 if kind == fq.NVFP4 else None, kind, 0))


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("size", PAST)
def test_rows_past_32_bits_are_refused(fq, kind, size):
    L, BF, small = fq.lib(), fq.DT_BF16, 32
    op = operand(fq, kind)
    for M, N, K in ((size, 16, small), (16, size, small), (16, 16, size)):
        assert L.fp4_gemm(op, op, A, BF, M, N, K, None) == INVALID
    for M, N, K in ((size, 16, small), (1, size, small), (16, size, small), (17, size, small), (1, 16, size)):
        need = L.fp4q_linear_workspace_size(kind, M, N, K)
        for amax in (None, A):
            assert L.fp4_linear(A, BF, K, op, M, N, K, amax, A, BF, A, need, None) == INVALID
    for M, N, K in ((size, 16, small), (16, size, small), (16, small, size)):
        need = L.fp4q_linear_train_workspace_size(kind, M, N, K)
        assert L.fp4_linear_train(A, A, A, BF, M, N, K, kind, A, A, A, BF, A, need, None) == INVALID
