"""The norm's and the experts' entry points without a GPU: argument checks
before any device work, sizes, and the plain definitions that the GPU tests
compare with, tied to torch's own casts and to the oracle."""
import ctypes

import numpy as np
import pytest
import torch

import experts_reference as ref
import oracle

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


def test_norm_refuses(fq):
    f, BF, F = fq.lib().fp8_rmsnorm, fq.DT_BF16, fq.DT_F32
    tile = fq.SCALE_TILE_1x128

    def call(x=A, ldx=64, r=None, ldr=64, dt=BF, w=A, wdt=F, eps=1e-6, T=4, C=64, h=None, ldh=64, y=A, ldy=64,
             scaling=tile, q=A, s=A, rstd=A):
        e = None if eps is None else ctypes.byref(ctypes.c_float(eps))
        return f(x, ldx, r, ldr, dt, w, wdt, e, T, C, h, ldh, y, ldy, scaling, q, s, rstd, None)
    assert call(dt=2) == INVALID and call(wdt=-1) == INVALID and call(T=-1) == INVALID and call(C=-1) == INVALID
    assert call(T=1 << 30) == INVALID and call(C=1 << 30, ldx=1 << 30, ldy=1 << 30) == INVALID
    assert call(eps=None) == INVALID and call(eps=-1e-6) == INVALID
    assert call(eps=float("nan")) == INVALID and call(eps=float("inf")) == INVALID
    assert call(r=A) == INVALID and call(h=A) == INVALID        # they come together
    assert call(q=None) == INVALID and call(s=None) == INVALID
    for scaling in (fq.SCALE_TENSOR, fq.SCALE_BLOCK_128x128, fq.SCALE_MX_1x32, -1, 9):
        assert call(scaling=scaling) == INVALID
    assert call(x=None) == INVALID and call(w=None) == INVALID
    assert call(ldx=63) == INVALID and call(ldy=63) == INVALID and call(r=A, h=A, ldh=1) == INVALID
    assert call(x=P(0x10001)) == MISALIGNED and call(y=P(0x10001)) == MISALIGNED
    assert call(w=P(0x10002)) == MISALIGNED and call(s=P(0x10002)) == MISALIGNED
    assert call(rstd=P(0x10002)) == MISALIGNED and call(r=P(0x10001), h=A) == MISALIGNED
    assert call(ldx=1 << 61) == INVALID


def test_norm_backward_refuses(fq):
    f, BF, F = fq.lib().fp8_rmsnorm_backward, fq.DT_BF16, fq.DT_F32
    size = fq.lib().fp8q_rmsnorm_backward_workspace_size
    need = size(4, 64)
    assert need == 456 * 64 * 4 and size(-1, 64) == 0 and size(4, -1) == 0 and size(1 << 30, 4) == 0

    def call(dy=A, ldd=64, h=A, ldh=64, dt=BF, w=A, wdt=F, rstd=A, r=None, ldr=64, T=4, C=64, dx=A, ldx=64, dw=A,
             ws=A, n=need):
        return f(dy, ldd, h, ldh, dt, w, wdt, rstd, r, ldr, T, C, dx, ldx, dw, ws, n, None)
    assert call(dt=2) == INVALID and call(wdt=2) == INVALID and call(T=-1) == INVALID and call(C=1 << 31) == INVALID
    for k in ("dy", "h", "w", "rstd", "dx"):
        assert call(**{k: None}) == INVALID
    assert call(ldd=63) == INVALID and call(ldh=63) == INVALID and call(ldx=63) == INVALID
    assert call(r=A, ldr=63) == INVALID
    assert call(ws=None) == WORKSPACE and call(n=need - 1) == WORKSPACE
    assert call(ws=P(0x10010)) == MISALIGNED
    for k in ("dy", "h", "dx", "r"):
        assert call(**{k: P(0x10001)}) == MISALIGNED
    assert call(w=P(0x10002)) == MISALIGNED and call(rstd=P(0x10002)) == MISALIGNED
    assert call(dw=P(0x10002)) == MISALIGNED


def struct(fq, q=0x10000, qs=0x20000, qt=0x30000, qts=0x40000, off=0x50000, rows=256, cols=64, groups=4, fmt=0):
    return fq._ExpertsStruct(q, qs, qt, qts, off, rows, cols, groups, fmt)


def test_sizes(fq):
    f = fq.lib().fp8q_experts_blocks
    assert f(0, 1, 1) == 1 and f(127, 3, 1) == 3 and f(128, 3, 1) == 4 and f(300, 3, 0) == 3 and f(387, 3, 0) == 6
    assert f(-1, 1, 1) == 0 and f(10, 0, 1) == 0 and f(10, 1025, 1) == 0 and f(10, 3, 0) == 0
    assert f(2 ** 31 - 1, 1, 1) == 0 and f(2 ** 31 - 1025, 1024, 1) == 0
    g = fq.lib().fp8q_experts_scale_bytes
    assert g(128, 128, 1, 0) == 512 and g(128, 144, 1, 1) == 2 * 2 * 512 and g(128, 0, 1, 1) == 0
    assert g(128, 24, 1, 1) == 0 and g(1 << 30, 1 << 30, 1, 1) == 0
    for rows, groups, ragged in ((0, 1, True), (1000, 7, True), (1001, 7, False), (128, 128, False)):
        assert f(rows, groups, ragged) == fq.experts_blocks(rows, groups, ragged)


def test_cast_refuses(fq):
    f, BF = fq.lib().fp8_quantize_experts, fq.DT_BF16

    def call(x=A, dt=BF, T=100, ld=64, index=A, **out):
        return f(x, dt, T, ld, index, ctypes.byref(struct(fq, **out)), None)
    assert f(A, BF, 100, 64, A, None, None) == INVALID
    assert call(dt=3) == INVALID and call(T=-1) == INVALID and call(T=2 ** 31) == INVALID
    assert call(x=None) == INVALID and call(ld=63) == INVALID
    assert call(index=None) == INVALID                      # 100 rows are not 256
    assert call(fmt=2) == INVALID and call(groups=0) == INVALID and call(groups=1025) == INVALID
    assert call(cols=40) == INVALID and call(rows=-1) == INVALID and call(rows=2 ** 31) == INVALID
    assert call(off=None, groups=3) == INVALID              # 256 rows do not divide by 3
    assert call(q=None) == INVALID and call(qts=None) == INVALID
    assert call(q=None, qs=None, qt=None, qts=None) == INVALID
    for k in ("q", "qs", "qt", "qts"):
        assert call(**{k: 0x10008}) == MISALIGNED
    assert call(off=0x50002) == MISALIGNED and call(index=P(0x10002)) == MISALIGNED
    assert call(x=P(0x10001)) == MISALIGNED


def test_products_refuse(fq):
    lib, BF = fq.lib(), fq.DT_BF16

    def call(name, a, b, y=A, out=BF):
        return getattr(lib, name)(ctypes.byref(a), ctypes.byref(b), y, out, None)
    x = lambda **k: struct(fq, **k)
    w = lambda **k: struct(fq, **dict(dict(off=None, rows=4 * 32), **k))     # N = 32, K = 64
    g = lambda **k: struct(fq, **dict(dict(cols=32), **k))
    assert lib.fp8_experts_fprop(None, ctypes.byref(w()), A, BF, None) == INVALID
    assert lib.fp8_experts_wgrad(ctypes.byref(g()), None, A, BF, None) == INVALID
    for name, a in (("fp8_experts_fprop", x), ("fp8_experts_dgrad", g)):
        assert call(name, a(), w(), out=5) == INVALID and call(name, a(), w(), y=None) == INVALID
        assert call(name, a(), w(), y=ODD) == MISALIGNED
        assert call(name, a(cols=48), w()) == INVALID                        # another contraction
        assert call(name, a(groups=3), w()) == INVALID and call(name, a(), w(groups=2)) == INVALID
        assert call(name, a(), w(off=0x50000)) == INVALID                    # ragged weights
        assert call(name, a(q=None, qs=None), w()) == INVALID                # not by rows
        assert call(name, a(), w(rows=4 * 24)) == INVALID                    # N % 16
        assert call(name, a(fmt=9), w()) == INVALID and call(name, a(), w(fmt=-1)) == INVALID
        assert call(name, a(qs=0x10008), w()) == MISALIGNED
    long = 1 << 28
    assert call("fp8_experts_fprop", x(rows=16, cols=long, groups=1), w(rows=16, cols=long, groups=1)) == INVALID
    assert call("fp8_experts_wgrad", g(rows=long, groups=1), x(rows=long, groups=1)) == INVALID
    assert call("fp8_experts_fprop", x(cols=0), w(cols=0)) == INVALID         # nothing to contract over
    assert call("fp8_experts_fprop", x(), w(q=None, qs=None)) == INVALID
    assert call("fp8_experts_dgrad", g(), w(qt=None, qts=None)) == INVALID
    f = "fp8_experts_wgrad"
    assert call(f, g(), x(), out=5) == INVALID and call(f, g(), x(), y=None) == INVALID
    assert call(f, g(), x(), y=ODD) == MISALIGNED
    assert call(f, g(rows=128), x()) == INVALID and call(f, g(groups=2), x()) == INVALID
    assert call(f, g(off=None), x()) == INVALID
    assert call(f, g(qt=None, qts=None), x()) == INVALID and call(f, g(), x(qt=None, qts=None)) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="valid arguments would reach a kernel on placeholder pointers")
def test_random_arguments_get_a_status_not_a_crash(fq):
    """Seeded random arguments to every new entry point: a documented status each,
    before any device work (no device here: ARCH 3 or CUDA 6 past the checks)."""
    import random
    rng = random.Random(77)
    pick = rng.choice
    sizes = [-1, 0, 1, 15, 16, 48, 128, 130, 4096, 1 << 30, 2 ** 31 - 1, 1 << 40, (1 << 62) + 16]
    small = [0, 16, 32, 48, 128, 256]
    ptrs = [None, P(0x10000), P(0x10000), P(0x10008), P(0x10001)]
    addr = lambda: getattr(pick(ptrs), "value", None)
    lib = fq.lib()

    def operand():
        s = sizes if rng.random() < 0.3 else small
        return fq._ExpertsStruct(addr(), addr(), addr(), addr(), addr(), pick(s), pick(s), pick([-1, 0, 1, 2, 4, 1024, 1025]),
                                 pick([0, 1, 0, 1, 2, -1]))
    seen = set()
    for _ in range(20000):
        s = sizes if rng.random() < 0.3 else small
        kind = rng.randrange(4)
        if kind == 0:
            eps = pick([None, ctypes.byref(ctypes.c_float(1e-6)), ctypes.byref(ctypes.c_float(-1.0))])
            rc = lib.fp8_rmsnorm(pick(ptrs), pick(s), pick(ptrs), pick(s), pick([0, 1, 2]), pick(ptrs), pick([0, 1, 3]), eps,
                                 pick(s), pick(s), pick(ptrs), pick(s), pick(ptrs), pick(s), pick([0, 1, 3, 7]), pick(ptrs),
                                 pick(ptrs), pick(ptrs), None)
        elif kind == 1:
            rc = lib.fp8_rmsnorm_backward(pick(ptrs), pick(s), pick(ptrs), pick(s), pick([0, 1, 2]), pick(ptrs), pick([0, 1, 3]),
                                          pick(ptrs), pick(ptrs), pick(s), pick(s), pick(s), pick(ptrs), pick(s), pick(ptrs),
                                          pick(ptrs), pick([0, 1 << 30, 1 << 40]), None)
        elif kind == 2:
            rc = lib.fp8_quantize_experts(pick(ptrs), pick([0, 1, 2]), pick(s), pick(s), pick(ptrs), ctypes.byref(operand()), None)
        else:
            f = pick([lib.fp8_experts_fprop, lib.fp8_experts_dgrad, lib.fp8_experts_wgrad])
            rc = f(ctypes.byref(operand()), ctypes.byref(operand()), pick(ptrs), pick([0, 1, 2]), None)
        assert rc in (0, 1, 2, 3, 4, 6), (kind, rc)
        seen.add((kind, rc))
    assert {(k, 6) for k in range(3)} <= seen   # some passed every check


def test_only_the_current_device_serves(fq, monkeypatch):
    class On:
        def __init__(self, device):
            self.device = device

        def get_device(self):
            return self.device
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 2, raising=False)
    fq._here(On(2), None, On(2))
    for bad in ((On(0),), (On(2), None, On(1))):
        with pytest.raises(ValueError):
            fq._here(*bad)


def test_struct_layout_matches_header(fq, tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src, exe = tmp_path / "sz.c", tmp_path / "sz"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fp8q.h"\nint main(void){printf("%zu %zu %zu %zu %d",'
                   ' sizeof(fp8q_experts), offsetof(fp8q_experts, offsets), offsetof(fp8q_experts, cols),'
                   ' offsetof(fp8q_experts, format), FP8Q_EXPERTS_MAX);return 0;}\n')
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), "-I", "/usr/local/cuda/include", str(src), "-o",
                    str(exe)], check=True)
    got = list(map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()))
    s = fq._ExpertsStruct
    assert got == [ctypes.sizeof(s), s.offsets.offset, s.cols.offset, s.format.offset, fq.EXPERTS_MAX]


# --------------------------------------------------------- the definitions

def test_e5m2_bytes_are_torchs():
    b = np.arange(256, dtype=np.uint8)
    v = ref.e5m2_value(b)
    np.testing.assert_array_equal(v, torch.from_numpy(b).view(torch.float8_e5m2).double().numpy())
    ok = np.isfinite(v)
    np.testing.assert_array_equal(ref.e5m2_byte(v[ok]), b[ok])


@pytest.mark.parametrize("fmt", [0, 1])
def test_mx_rows_are_the_oracles(fmt):
    r = np.random.default_rng(1)
    x = (r.standard_normal((256, 128)) * np.exp(r.uniform(-30, 30, (256, 1)))).astype(np.float32)
    x[3, 4], x[5, 40], x[7] = np.nan, np.inf, 0.0
    q, scales = oracle.quantize_mx_rows(x, fmt)
    b, code = ref.mx_rows(x.astype(np.float64), fmt)
    np.testing.assert_array_equal(b, q)
    np.testing.assert_array_equal(code, scales.reshape(code.shape))


def test_groups_never_meet():
    """Every group's blocks end before the next group's begin, and inside the operand."""
    r = np.random.default_rng(2)
    for _ in range(300):
        E = int(r.integers(1, 40))
        sizes = r.integers(0, r.integers(1, 400), E)
        ends = [0] + np.cumsum(sizes).tolist()
        S = ends[-1] + int(r.integers(0, 200))
        last = 0
        for _, a, z, b in ref.Groups(ends):
            assert b >= last
            last = b + -(-(z - a) // 128)
        assert last <= S // 128 + E


def test_norm_is_torchs():
    h, w = torch.randn(5, 70, dtype=torch.float64), torch.randn(70, dtype=torch.float64)
    _, y = ref.norm(h.numpy(), w.numpy(), 1e-5)
    np.testing.assert_allclose(y, torch.nn.functional.rms_norm(h, (70,), w, 1e-5).numpy(), rtol=1e-12)
    h.requires_grad_(), w.requires_grad_()
    dy, dres = torch.randn(5, 70, dtype=torch.float64), torch.randn(5, 70, dtype=torch.float64)
    (torch.nn.functional.rms_norm(h, (70,), w, 1e-5) * dy + dres * h).sum().backward()
    rstd = 1 / np.sqrt((h.detach().numpy() ** 2).mean(axis=1) + 1e-5)
    dx, dw, _, _ = ref.norm_backward(dy.numpy(), h.detach().numpy(), w.detach().numpy(), rstd, dres.numpy())
    np.testing.assert_allclose(dx, h.grad.numpy(), rtol=1e-9, atol=1e-12)
    np.testing.assert_allclose(dw, w.grad.numpy(), rtol=1e-9, atol=1e-12)
