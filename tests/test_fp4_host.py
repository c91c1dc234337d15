"""The 4-bit and activation-checkpoint entry points without a GPU: argument
checks before any device work, workspace sizes, and the plain definitions the
GPU tests compare with, tied to torch's own casts."""
import ctypes

import numpy as np
import pytest
import torch

import fp4_reference as ref

P = ctypes.c_void_p
A, ODD = P(0x10000), P(0x10008)
INVALID, MISALIGNED, WORKSPACE = 1, 2, 4


@pytest.fixture(scope="module")
def fq():
    from scaled_quantize_fp8_warp_gb300 import build_lib
    import scaled_quantize_fp8_warp_gb300 as fq
    build_lib.build()
    fq.load_library()
    return fq


def operand(fq, kind, data=0x10000, scales=0x20000, g="fit", reserved=0):
    if g == "fit":
        g = 0x30000 if kind == fq.NVFP4 else None
    return ctypes.byref(fq._Fp4Struct(data, scales, g, kind, reserved))


def test_scale_bytes(fq):
    f = fq.lib().fp4q_scale_bytes
    assert f(fq.MXFP4, 128, 128) == 512 and f(fq.MXFP4, 129, 129) == 4 * 512
    assert f(fq.NVFP4, 128, 128) == 2 * 512 and f(fq.NVFP4, 1, 1) == 512
    assert f(fq.MXFP4, 0, 5) == 0 and f(2, 128, 128) == 0 and f(fq.MXFP4, -1, 128) == 0
    assert f(fq.MXFP4, 1 << 40, 1 << 40) == 0


def test_quantize_refuses(fq):
    f = fq.lib().fp4_quantize
    MX, NV, BF = fq.MXFP4, fq.NVFP4, fq.DT_BF16

    def call(x=A, dt=BF, r=4, c=64, ld=64, kind=MX, amax=None, q=A, qs=A, qt=None, qts=None, g=None):
        return f(x, dt, r, c, ld, kind, amax, q, qs, qt, qts, g, None)
    assert call(dt=5) == INVALID and call(kind=2) == INVALID and call(r=-1) == INVALID
    assert call(ld=63) == INVALID                       # rows overlap
    assert call(x=None) == INVALID
    assert call(q=None) == INVALID                      # half a pair
    assert call(q=None, qs=None) == INVALID             # no output
    assert call(kind=NV) == INVALID                     # no amax, no tensor scale
    assert call(kind=NV, amax=A) == INVALID and call(kind=NV, g=A) == INVALID
    assert call(g=A) == INVALID                         # MXFP4 has no tensor scale
    assert call(x=P(0x10001)) == MISALIGNED             # not aligned to bf16
    assert call(q=ODD) == MISALIGNED and call(qt=A, qts=ODD) == MISALIGNED
    assert call(kind=NV, amax=P(0x10002), g=A) == MISALIGNED
    assert call(r=1 << 40, c=1 << 40, ld=1 << 40) == INVALID


def test_dequantize_and_gemm_refuse(fq):
    MX, NV, BF = fq.MXFP4, fq.NVFP4, fq.DT_BF16
    f = fq.lib().fp4_dequantize
    assert f(None, 4, 64, A, BF, None) == INVALID
    assert f(operand(fq, 2), 4, 64, A, BF, None) == INVALID
    assert f(operand(fq, MX, g=0x30000), 4, 64, A, BF, None) == INVALID
    assert f(operand(fq, NV, g=None), 4, 64, A, BF, None) == INVALID
    assert f(operand(fq, MX, reserved=1), 4, 64, A, BF, None) == INVALID
    assert f(operand(fq, MX, data=0x10008), 4, 64, A, BF, None) == MISALIGNED
    assert f(operand(fq, MX), 4, 64, ODD, BF, None) == MISALIGNED
    assert f(operand(fq, MX), 4, 64, A, 7, None) == INVALID
    g = fq.lib().fp4_gemm
    assert g(operand(fq, MX), operand(fq, NV), A, BF, 4, 4, 64, None) == INVALID
    assert g(operand(fq, MX), operand(fq, MX), None, BF, 4, 4, 64, None) == INVALID
    assert g(operand(fq, MX), operand(fq, MX), ODD, BF, 4, 4, 64, None) == MISALIGNED
    assert g(operand(fq, MX), operand(fq, MX), A, BF, 4, -4, 64, None) == INVALID
    assert g(operand(fq, MX), operand(fq, MX), A, BF, 1 << 40, 1 << 40, 64, None) == INVALID


def test_linear_refuses(fq):
    MX, NV, BF = fq.MXFP4, fq.NVFP4, fq.DT_BF16
    L = fq.lib()
    need = L.fp4q_linear_workspace_size(NV, 5, 64, 96)
    assert need == 256 + 256 + 1024 and L.fp4q_linear_workspace_size(9, 5, 64, 96) == 0
    assert L.fp4q_linear_workspace_size(NV, 1 << 40, 64, 1 << 40) == 0

    def call(ld=96, w=None, ws=A, n=need, y=A, amax=None, dt=BF):
        return L.fp4_linear(A, dt, ld, w or operand(fq, NV), 5, 64, 96, amax, y, BF, ws, n, None)
    assert call(ld=95) == INVALID and call(dt=3) == INVALID and call(y=None) == INVALID
    assert call(n=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(ws=P(0x10010)) == MISALIGNED and call(amax=P(0x10001)) == MISALIGNED
    t = L.fp4_linear_train
    need = L.fp4q_linear_train_workspace_size(MX, 5, 64, 96)
    assert need > 0 and L.fp4q_linear_train_workspace_size(MX, -5, 64, 96) == 0
    args = lambda dw=A, kind=MX, n=need: (A, A, A, BF, 5, 64, 96, kind, A, A, dw, BF, A, n, None)
    assert t(*args(dw=None)) == INVALID and t(*args(kind=3)) == INVALID
    assert t(*args(n=need - 1)) == WORKSPACE and t(*args(dw=ODD)) == MISALIGNED


def test_act_refuses(fq):
    L = fq.lib()
    BF = fq.DT_BF16

    def fwd(act=0, dt=BF, T=4, F=64, u=A, ldu=64, v=A, ldv=64, a=A, lda=64, u8=A, us=A, v8=A, vs=A):
        return L.fp8_act_forward(act, dt, T, F, u, ldu, v, ldv, a, lda, u8, us, v8, vs, None)
    assert fwd(act=3) == INVALID and fwd(act=-1) == INVALID and fwd(dt=2) == INVALID
    assert fwd(ldu=63) == INVALID and fwd(ldv=63) == INVALID and fwd(lda=63) == INVALID
    assert fwd(v=None) == INVALID and fwd(v8=None) == INVALID and fwd(vs=None) == INVALID
    assert fwd(u8=None) == INVALID and fwd(us=None) == INVALID and fwd(T=-1) == INVALID
    assert fwd(u=P(0x10001)) == MISALIGNED and fwd(us=P(0x10002)) == MISALIGNED
    assert fwd(vs=P(0x10002)) == MISALIGNED

    def bwd(u8=A, us=A, v8=A, vs=A, da=A, ldda=64, du=A, dv=A, a=None, lda=0):
        return L.fp8_act_backward(0, BF, 4, 64, u8, us, v8, vs, da, ldda, du, 64, dv, 64, a, lda,
                                  None)
    assert bwd(vs=None) == INVALID and bwd(dv=None) == INVALID and bwd(v8=None) == INVALID
    assert bwd(da=None) == INVALID and bwd(ldda=10) == INVALID and bwd(du=None) == INVALID
    assert bwd(a=A, lda=10) == INVALID and bwd(du=P(0x10001)) == MISALIGNED


def test_binding_refuses(fq):
    """Shapes and types the C entry points cannot see."""
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fq.Fp4Operand(u8(4, 16), u8(512), fq.MXFP4, 64)          # 64 codes take 32 bytes
    with pytest.raises(ValueError):
        fq.Fp4Operand(u8(4, 32), u8(511), fq.MXFP4, 64)
    with pytest.raises(ValueError):
        fq.Fp4Operand(u8(4, 32), u8(512), fq.NVFP4, 64)          # no tensor scale
    with pytest.raises(ValueError):
        fq.Fp4Operand(u8(4, 32), u8(512), fq.MXFP4, 64, torch.ones(1))
    with pytest.raises(ValueError):
        fq.ActCheckpoint(u8(4, 200), torch.zeros(1, 4))          # two tiles a row
    with pytest.raises(ValueError):
        fq.ActCheckpoint(u8(4, 200), torch.zeros(2, 4), u8(4, 200))
    with pytest.raises(ValueError):
        fq.fp8_act_forward(fq.ACT_SILU, torch.zeros(4, 8))       # not on a GPU
    with pytest.raises(ValueError):
        fq.fp4_quantize(torch.zeros(4, 8), fq.MXFP4)


# ------------------------------------------- the plain definitions themselves

def test_reference_e4m3_is_torchs():
    b = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(b).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(ref.e4m3_value(b), t.astype(np.float64))
    v = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * 30
    q = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.e4m3_byte(np.copysign(ref.round_float(v, 3, -6, 448), v)), q)


def test_reference_e2m1_rounds_to_the_nearest_and_to_even():
    v = np.random.default_rng(1).uniform(-8, 8, 20000)
    got = ref.E2M1[ref.e2m1_code(v)]
    near = np.abs(v[:, None] - ref.E2M1[None, :]).min(1)
    np.testing.assert_allclose(np.abs(v - got), near, rtol=0, atol=0)
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert ref.E2M1[ref.e2m1_code(np.array(ties))].tolist() == [0, 1, 1, 2, 2, 4, 4]
    assert ref.e2m1_code(np.array([-0.0, 0.0, 1e9, -1e9])).tolist() == [8, 0, 7, 15]


def test_reference_quantize_by_hand():
    x = np.zeros((1, 64), np.float32)
    x[0, :3] = [7.0, -3.0, 1.2]                  # amax 7: scale 1, 7 saturates at 6
    x[0, 32:34] = [24.0, 3.0]                    # amax 24: scale 4
    codes, byte, _ = ref.quantize(x, 0)
    assert byte.tolist() == [[127, 129]]
    assert ref.values(codes, byte, None, 0, 64)[0, [0, 1, 2, 32, 33]].tolist() == [6, -3, 1, 24, 4]
    x[0, 16] = 0.5
    codes, byte, g = ref.quantize(x, 1)
    assert g == np.float32(24) / np.float32(2688)
    # 7/6 and 0.5/6 over g are 130.67 and 9.33: E4M3 128 and 9
    assert ref.e4m3_value(byte).tolist() == [[128, 9, 448, 2.0 ** -9]]


def test_reference_gradients_are_the_differences():
    u = np.linspace(-6, 6, 97)
    h = 1e-5
    for name in ("silu", "gelu", "gelu_tanh"):
        d = (ref.act(name, u + h) - ref.act(name, u - h)) / (2 * h)
        np.testing.assert_allclose(ref.act_grad(name, u), d, rtol=0, atol=1e-9)
