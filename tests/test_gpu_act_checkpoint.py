"""Activation functions with 8-bit checkpoints on the GPU against plain 64-bit
definitions: checkpoints bit for bit, results within act_bound / grad_bound
plus the output's rounding."""
import numpy as np
import pytest
import torch

import fp4_reference as ref

pytestmark = pytest.mark.gpu
ACTS = ["silu", "gelu", "gelu_tanh"]
SHAPES = [(1, 1), (1, 16), (1, 16384), (2, 128), (3, 130), (7, 1000), (33, 257), (64, 1024)]


@pytest.fixture(scope="module")
def fq():
    import scaled_quantize_fp8_warp_gb300 as fq
    yield fq
    assert fq.device_status() == fq.OK


def normal(shape, seed, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def f32(t):
    return t.detach().float().cpu().numpy()


def code(fq, name):
    return {"silu": fq.ACT_SILU, "gelu": fq.ACT_GELU, "gelu_tanh": fq.ACT_GELU_TANH}[name]


def near(got, want, bound, what):
    """Within `bound` and the rounding of got's type."""
    eps = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -23
    err = np.abs(f64(got) - want)
    bad = err > bound + eps * np.abs(want) + 1e-37
    assert not bad.any(), (what, bad.sum(), np.argwhere(bad)[:3], err.max())


def check_saved(fq, q, s, x, what):
    want_q, want_s = ref.save(f32(x))
    np.testing.assert_array_equal(s.cpu().numpy(), want_s, err_msg=what)
    np.testing.assert_array_equal(q.cpu().numpy(), want_q, err_msg=what)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(fq, name, gated, dtype, shape):
    u = normal(shape, 1, 2.5, dtype)
    v = normal(shape, 2, 1.0, dtype) if gated else None
    a, kept = fq.fp8_act_forward(code(fq, name), u.cuda(), v.cuda() if gated else None)
    check_saved(fq, kept.u, kept.u_scales, u, "u")
    w = f64(v) if gated else 1.0
    if gated:
        check_saved(fq, kept.v, kept.v_scales, v, "v")
    else:
        assert kept.v is None
    near(a, ref.act(name, f64(u)) * w, ref.act_bound(f64(u)) * np.abs(w), "a")


def check_backward(fq, name, kept, da, want_a, got):
    du, dv, a = got
    u = ref.saved(kept.u.cpu().numpy(), kept.u_scales.cpu().numpy())
    gated = kept.v is not None
    v = ref.saved(kept.v.cpu().numpy(), kept.v_scales.cpu().numpy()) if gated else 1.0
    u32 = 2.0 ** -23 * np.abs(u)     # the held value is rounded to fp32: moves f by |f'| <= 1.2 of it
    f, df = ref.act(name, u), ref.act_grad(name, u)
    d = f64(da)
    near(du, d * v * df, np.abs(d * v) * (ref.grad_bound(u) + u32), "du")
    if gated:
        near(dv, d * f, np.abs(d) * (ref.act_bound(u) + 2 * u32), "dv")
    else:
        assert dv is None
    if want_a:
        near(a, f * v, np.abs(v) * (ref.act_bound(u) + 2 * u32), "a")
    else:
        assert a is None


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(fq, name, gated, dtype, shape):
    u, v = normal(shape, 3, 2.5), normal(shape, 4) if gated else None
    _, kept = fq.fp8_act_forward(code(fq, name), u.cuda(), v.cuda() if gated else None)
    da = normal(shape, 5, 1e-2, dtype)
    for want_a in (False, True):
        got = fq.fp8_act_backward(code(fq, name), kept, da.cuda(), want_a=want_a)
        check_backward(fq, name, kept, da, want_a, got)


@pytest.mark.parametrize("name", ACTS)
def test_gradient_is_the_difference_of_the_forward(fq, name):
    """du and dv against central differences, in 64 bits, of sum(f(u) v) at the
    values the checkpoint holds."""
    shape = (9, 300)
    _, kept = fq.fp8_act_forward(code(fq, name), normal(shape, 6, 2.0, torch.float32).cuda(),
                                 normal(shape, 7, 1.0, torch.float32).cuda())
    du, dv, a = fq.fp8_act_backward(code(fq, name), kept, torch.ones(shape, device="cuda"), want_a=True)
    u = ref.saved(kept.u.cpu().numpy(), kept.u_scales.cpu().numpy())
    v = ref.saved(kept.v.cpu().numpy(), kept.v_scales.cpu().numpy())
    h = 1e-5     # the difference is off by h^2 / 6 |f'''| < 1e-10, its rounding by 1e-10
    diff = v * (ref.act(name, u + h) - ref.act(name, u - h)) / (2 * h)
    slack = 2.0 ** -23 * (1 + np.abs(u))
    assert (np.abs(f64(du) - diff) <= np.abs(v) * (ref.grad_bound(u) + slack) + 1e-9).all()
    assert (np.abs(f64(dv) - ref.act(name, u)) <= ref.act_bound(u) + 2 * slack * np.abs(u)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_checkpoint_is_the_tile_quantizers(fq, dtype):
    u, v = normal((200, 1040), 8, 3.0, dtype).cuda(), normal((200, 1040), 9, 1e-3, dtype).cuda()
    u[3, 5], u[4, 700], v[5, 1039], v[6, 0] = float("nan"), float("inf"), float("-inf"), -float("nan")
    v[7] = 0.0
    v[8] = -0.0
    _, kept = fq.fp8_act_forward(fq.ACT_SILU, u, v)
    for x, q, s in ((u, kept.u, kept.u_scales), (v, kept.v, kept.v_scales)):
        want, want_s, _, _ = fq.fp8_quantize_tile1x128(x, fq.E4M3)
        assert torch.equal(q, want)
        assert torch.equal(s.nan_to_num(7.0), want_s.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("F,ld", [(256, 512), (250, 513), (100, 208), (16, 40)])
def test_halves_of_one_matrix_and_rows_apart(fq, dtype, F, ld):
    T = 21
    h = normal((T, ld), 10, 2.0, dtype).cuda()
    u, v = h[:, :F], h[:, ld - F:]
    wide = torch.full((T, F + 9), 7.0, dtype=dtype, device="cuda")
    a, kept = fq.fp8_act_forward(fq.ACT_GELU, u, v, out=wide[:, 3:3 + F])
    b, kept2 = fq.fp8_act_forward(fq.ACT_GELU, u.contiguous(), v.contiguous())
    assert torch.equal(a, b) and torch.equal(kept.u, kept2.u) and torch.equal(kept.v, kept2.v)
    assert (wide[:, :3] == 7).all() and (wide[:, 3 + F:] == 7).all()
    dh = torch.full((T, ld), 5.0, dtype=dtype, device="cuda")
    da = normal((T, F + 4), 11, 1.0, dtype).cuda()[:, 1:1 + F]
    fq.fp8_act_backward(fq.ACT_GELU, kept, da, du=dh[:, :F], dv=dh[:, ld - F:])
    du, dv, _ = fq.fp8_act_backward(fq.ACT_GELU, kept, da.contiguous())
    assert torch.equal(dh[:, :F], du) and torch.equal(dh[:, ld - F:], dv)
    assert (dh[:, F:ld - F] == 5).all()


def test_in_place(fq):
    u, v = normal((37, 640), 12).cuda(), normal((37, 640), 13).cuda()
    a, kept = fq.fp8_act_forward(fq.ACT_SILU, u, v)
    w = u.clone()
    fq.fp8_act_forward(fq.ACT_SILU, w, v, out=w)
    assert torch.equal(w, a)
    da = normal((37, 640), 14).cuda()
    du, dv, _ = fq.fp8_act_backward(fq.ACT_SILU, kept, da)
    d = da.clone()
    fq.fp8_act_backward(fq.ACT_SILU, kept, d, du=d)
    assert torch.equal(d, du)


@pytest.mark.parametrize("name", ACTS)
def test_large_inputs_stay_finite(fq, name):
    big = torch.tensor([-3e38, -1e30, -1e10, -200.0, -88.0, -20.0, 0.0, -0.0, 20.0, 88.0, 200.0, 1e10,
                        1e30, 3e38, 1e-38, -1e-40], device="cuda")
    u = torch.zeros((16, 128), device="cuda")
    u[:, 0] = big            # a tile of its own each: the checkpoint keeps it to 4 bits
    a, kept = fq.fp8_act_forward(code(fq, name), u)
    want = torch.where(big > 30, big, torch.zeros_like(big))
    far = big.abs() >= 88
    assert torch.isfinite(a).all() and torch.allclose(a[far, 0], want[far], rtol=1e-6, atol=1e-30)
    du, _, _ = fq.fp8_act_backward(code(fq, name), kept, torch.ones_like(u))
    assert torch.isfinite(du).all()
    assert torch.allclose(du[far, 0], (big > 0).float()[far], rtol=1e-6, atol=1e-30)


def test_zero_sizes(fq):
    for shape in ((0, 64), (5, 0)):
        u = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        a, kept = fq.fp8_act_forward(fq.ACT_SILU, u, u)
        du, dv, b = fq.fp8_act_backward(fq.ACT_SILU, kept, u, want_a=True)
        assert a.shape == du.shape == dv.shape == b.shape == shape


def test_another_stream(fq):
    u, v = normal((500, 2048), 15).cuda(), normal((500, 2048), 16).cuda()
    a, kept = fq.fp8_act_forward(fq.ACT_GELU_TANH, u, v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, kept2 = fq.fp8_act_forward(fq.ACT_GELU_TANH, u, v, stream=s)
    got = fq.fp8_act_backward(fq.ACT_GELU_TANH, kept2, u, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, b) and torch.equal(kept.u, kept2.u)
    assert torch.equal(got[0], fq.fp8_act_backward(fq.ACT_GELU_TANH, kept, u)[0])


def test_offsets_past_32_bits(fq):
    T, F = 140000, 16400
    u = torch.zeros((T, F), dtype=torch.bfloat16, device="cuda")
    u[-5:] = normal((5, F), 17, 2.0).cuda()
    a, kept = fq.fp8_act_forward(fq.ACT_SILU, u)
    b, alone = fq.fp8_act_forward(fq.ACT_SILU, u[-5:].contiguous())
    assert torch.equal(a[-5:], b) and torch.equal(kept.u[-5:], alone.u)
    assert torch.equal(kept.u_scales[:, -5:], alone.u_scales)
    du, _, _ = fq.fp8_act_backward(fq.ACT_SILU, kept, u)
    want, _, _ = fq.fp8_act_backward(fq.ACT_SILU, alone, u[-5:].contiguous())
    assert torch.equal(du[-5:], want)
