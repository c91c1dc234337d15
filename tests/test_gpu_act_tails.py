"""Activation functions and their derivatives where they are small: relative
to their own value (or their terms'), not to 1, against 64 bits.

Bounds, in units of 2^-23, before any run.  The base-2 exponential's argument
a (|a| = 1.443 |u| for SiLU, 0.721 u^2 for GELU, u (2.302 + 0.103 u^2) for the
tanh form) carries at most three roundings and two rounded constants, 1.5 |a|
of the exponential in all; the exponential, the sum with 1, a reciprocal, GELU's
fitted factor (2.7) and the last products add at most 8.  A difference 1 - p
adds 2 of p.  Results below 2^-126 times |u| may be flushed to zero."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ACTS = ["silu", "gelu", "gelu_tanh"]
LOWEST = {"silu": -87.0, "gelu": -13.5, "gelu_tanh": -9.5}
ULP, TINY = 2.0 ** -23, 2e-36
_erfc = np.vectorize(math.erfc)


@pytest.fixture(scope="module")
def fq():
    import scaled_quantize_fp8_warp_gb300 as fq
    yield fq
    assert fq.device_status() == fq.OK


def parts(name, u):
    """p with f = u p, 1 - p, |a|, and the factor of u in f' = p + u (...)."""
    if name == "gelu":
        return (0.5 * _erfc(-u / math.sqrt(2)), 0.5 * _erfc(u / math.sqrt(2)), 0.7214 * u * u,
                np.exp(-u * u / 2) / math.sqrt(2 * math.pi))
    z = u if name == "silu" else 2 * math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)
    dz = 1.0 if name == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * u * u)
    p, r = 1 / (1 + np.exp(-z)), 1 / (1 + np.exp(z))
    return p, r, 1.4427 * np.abs(z), p * r * dz


def column(name, dtype):
    """Inputs one to a row, so that each is a checkpoint tile of its own."""
    u = torch.cat([torch.linspace(LOWEST[name], 12.0, 3000, dtype=torch.float64),
                   -torch.logspace(-6, math.log10(-LOWEST[name]), 500, dtype=torch.float64),
                   torch.tensor([-4.0, -5.0, -5.5, -6.0, -8.0, -9.0, -12.0]).double().clamp(min=LOWEST[name])])
    return u.to(dtype).view(-1, 1).cuda()


def near(got, want, bound, what):
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else ULP    # one rounding of the output, doubled
    err = np.abs(got.double().cpu().numpy() - want)
    bad = err > bound + half * np.abs(want) + TINY
    assert not bad.any(), (what, bad.sum(), np.argwhere(bad)[:3], (err / (np.abs(want) + TINY)).max())


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gated", [False, True])
def test_forward_keeps_its_digits(fq, name, dtype, gated):
    act = {"silu": fq.ACT_SILU, "gelu": fq.ACT_GELU, "gelu_tanh": fq.ACT_GELU_TANH}[name]
    u = column(name, dtype)
    v = torch.linspace(0.5, 2.0, u.numel()).to(dtype).view(-1, 1).cuda() if gated else None
    a, _ = fq.fp8_act_forward(act, u, v)
    x = u.double().cpu().numpy()
    p, _, arg, _ = parts(name, x)
    f = x * p * (v.double().cpu().numpy() if gated else 1.0)
    near(a, f, (8 + 1.5 * arg) * ULP * np.abs(f), name)


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward_keeps_its_digits(fq, name, dtype):
    act = {"silu": fq.ACT_SILU, "gelu": fq.ACT_GELU, "gelu_tanh": fq.ACT_GELU_TANH}[name]
    _, kept = fq.fp8_act_forward(act, column(name, torch.float32), column(name, torch.float32).abs() + 1)
    value = lambda q, s: (q.view(torch.float8_e4m3fn).float() * s.t()).double().cpu().numpy()
    x, w = value(kept.u, kept.u_scales), value(kept.v, kept.v_scales)
    du, dv, a = fq.fp8_act_backward(act, kept, torch.ones(x.shape, dtype=dtype, device="cuda"), want_a=True)
    p, r, arg, slope = parts(name, x)
    rel = (8 + 1.5 * arg) * ULP
    f, df = x * p, p + x * slope
    near(dv, f, rel * np.abs(f), name + " dv")
    near(a, f * w, (rel + ULP) * np.abs(f * w), name + " a")
    # 1 - p is a difference for the logistic forms alone
    lost = 0.0 if name == "gelu" else 2 * ULP * np.abs(x) * p * (slope / (p * r))
    near(du, df * w, (rel * (p + np.abs(x) * slope) + lost) * w + 2 * ULP * np.abs(df * w), name + " du")


def test_gelu_below_minus_5_5_is_not_zero(fq):
    u = torch.tensor([[-5.6], [-6.0], [-8.0], [-10.0]], device="cuda")
    a, _ = fq.fp8_act_forward(fq.ACT_GELU, u)
    assert (a < 0).all()
