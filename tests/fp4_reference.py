"""Plain definitions, in numpy with 64-bit arithmetic, of the 4-bit formats and
of the activation functions with 8-bit checkpoints.  Where a definition rounds
to fp32 (a held scale, a quotient), so does this."""
import math

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
BLOCK = {0: 32, 1: 16}
ATOM_K = {0: 128, 1: 64}


def round_float(v, frac_bits, min_exp, top):
    """Nearest (ties to even) float with `frac_bits` fraction bits, exponents
    from min_exp (subnormals below), clipped at +-top.  NaN stays NaN."""
    v = np.asarray(v, np.float64)
    with np.errstate(all="ignore"):
        e = np.maximum(np.frexp(v)[1] - 1, min_exp)
        step = np.ldexp(1.0, e - frac_bits)
        r = np.where(np.isinf(v), v, np.rint(v / step) * step)
        return np.clip(r, -top, top)


def e4m3_byte(v):
    """Byte of an E4M3 value (finite, representable)."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    e = np.maximum(np.frexp(a)[1] - 1, -6)
    m = a / np.ldexp(1.0, e - 3)                      # 0..15
    code = np.where(m >= 8, (e + 7) * 8 + (m - 8), m)
    return (code + 128 * np.signbit(v)).astype(np.uint8)


def e4m3_value(b):
    b = np.asarray(b, np.uint8).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e > 0, np.ldexp(1.0 + m / 8, e - 7), np.ldexp(m / 8.0, -6))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


def e2m1_code(v):
    """Code of RNE, saturating; the sign bit is v's."""
    r = np.abs(round_float(v, 1, 0, 6.0))
    code = np.searchsorted(E2M1[:8], r)
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def nv_global(amax):
    g = np.float32(np.float32(amax) / np.float32(2688))
    return np.float32(1e-12) if g < np.float32(1e-12) else g


def quantize(x, kind, amax=None):
    """x [R, C] fp32 -> (codes [R, Kp] uint8, scale bytes [R, blocks] uint8, g);
    Kp = C rounded up to 32, blocks = ceil(C / block)."""
    R, C = x.shape
    n = BLOCK[kind]
    t = np.zeros((R, -(-C // n) * n), np.float32)
    t[:, :C] = x
    t = t.reshape(R, -1, n)
    with np.errstate(all="ignore"):
        top = np.where(np.isnan(t).any(2), np.float32(np.nan), np.abs(t).max(2, initial=0))
        finite = np.isfinite(top)
        safe = np.where(finite, top, 0).astype(np.float32)
        if kind == 0:
            g = None
            code = np.where(safe > 0, np.frexp(safe)[1] - 1 - 2 + 127, 0)
            code = np.where(safe < np.float32(2.0 ** -126), 0, np.clip(code, 0, 254))
            byte = np.where(finite, code, 255).astype(np.uint8)
            d = np.ldexp(1.0, code - 127)
        else:
            if amax is None:
                amax = np.abs(x).max(initial=0) if not np.isnan(x).any() else np.nan
            g = nv_global(amax)
            finite &= bool(np.isfinite(g))
            s = (safe / np.float32(6)).astype(np.float32) / g
            s = np.maximum(round_float(np.where(np.isfinite(s), s, 448), 3, -6, 448.0), 2.0 ** -9)
            byte = np.where(finite, e4m3_byte(s), 0x7F).astype(np.uint8)
            d = (s.astype(np.float32) * (g if np.isfinite(g) else np.float32(1))).astype(np.float32)
        q = t.astype(np.float64) / d[..., None] if kind == 0 else \
            (t / d.astype(np.float32)[..., None]).astype(np.float64)
        codes = np.where(finite[..., None], e2m1_code(np.nan_to_num(q, nan=0.0)), 0)
    out = np.zeros((R, -(-C // 32) * 32), np.uint8)
    out[:, :codes.shape[1] * n][:, :t.shape[1] * n] = codes.reshape(R, -1)
    out[:, C:] = 0
    return out, byte, g


def pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def atoms(byte, kind, rows, K):
    """Scale bytes in the atom layout, zero past the matrix."""
    blocks = byte.shape[1]
    nk, nr = -(-K // ATOM_K[kind]), -(-rows // 128)
    out = np.zeros((nr * nk * 512,), np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(blocks), indexing="ij")
    at = ((r // 128) * nk + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    out[at.reshape(-1)] = byte.reshape(-1)
    return out


def values(codes, byte, g, kind, K):
    """What an operand stands for, in float64: code * scale, the NVFP4 scale
    s g rounded to fp32."""
    if kind == 0:
        s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    else:
        with np.errstate(all="ignore"):
            s = (e4m3_value(byte).astype(np.float32) * g).astype(np.float64)
    v = E2M1[codes[:, :K]]
    return v * np.repeat(s, BLOCK[kind], axis=1)[:, :K]


def dequantized(x, kind, amax=None):
    codes, byte, g = quantize(x, kind, amax)
    return values(codes, byte, g, kind, x.shape[1])


def product_bound(a, b, bf16):
    """|C - a b^T| allowed: the accumulator drops what lies below its last
    place, at most 2^-23 of the partial sum, once per 64-wide step, and once
    more for each of the tensor scales and a join of partial sums; then half a
    spacing of the output (2^-24 or 2^-9 relative, doubled for a tie on the
    other side)."""
    mag = np.abs(a) @ np.abs(b).T
    return (a.shape[1] / 64 + 12) * 2.0 ** -23 * mag + \
        (2.0 ** -8 if bf16 else 2.0 ** -23) * np.abs(a @ b.T)


def save(x):
    """E4M3 bytes under 1x128 tile scales: (bytes [T, F], scales [tiles, T])."""
    T, F = x.shape
    t = np.zeros((T, -(-F // 128) * 128), np.float32)
    t[:, :F] = x
    t = t.reshape(T, -1, 128)
    top = np.abs(t).max(2)
    s = np.maximum((top / np.float32(448)).astype(np.float32), np.float32(1e-12))
    q = (t / s[..., None]).astype(np.float32).astype(np.float64)
    b = e4m3_byte(np.copysign(np.abs(round_float(q, 3, -6, 448.0)), t))
    return b.reshape(T, -1)[:, :F], np.ascontiguousarray(s.T)


def saved(b, s):
    return e4m3_value(b) * np.repeat(s.T.astype(np.float64), 128, axis=1)[:, :b.shape[1]]


_erf = np.vectorize(math.erf)


def act(name, u):
    """f(u) in float64."""
    if name == "silu":
        return u / (1 + np.exp(-u))
    if name == "gelu":
        return 0.5 * u * (1 + _erf(u / math.sqrt(2)))
    return 0.5 * u * (1 + np.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))


def act_grad(name, u):
    if name == "silu":
        s = 1 / (1 + np.exp(-u))
        return s * (1 + u * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + _erf(u / math.sqrt(2))) + u * np.exp(-u * u / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = np.tanh(c * (u + 0.044715 * u ** 3))
    return 0.5 * (1 + t) + 0.5 * u * (1 - t * t) * c * (1 + 3 * 0.044715 * u * u)


def act_bound(u):
    """|f - f(u)| allowed for fp32 arithmetic.  The base-2 exponential is good
    to 2 + 1.16 |x| units in the last place and its argument x (|x| <= 2 |z|
    of tanh, at most 2 |u| + 0.08 |u|^3) carries three roundings, so f's factor
    is off by at most (8 + 4 |x|) 2^-23 of itself, or, where it is a difference
    from 1 (erf), by that much absolutely."""
    x = np.minimum(2 * np.abs(u) + 0.08 * np.abs(u) ** 3, 90)
    return (8 + 4 * x) * 2.0 ** -23 * np.abs(u) * np.minimum(1, np.exp(u) + 2.0 ** -1)


def grad_bound(u):
    """The same for f'(u): a sum of terms of at most 1 + |u| (1 + 0.14 u^2),
    each within act_bound's relative error, the last damped like e^-|u|."""
    x = np.minimum(2 * np.abs(u) + 0.08 * np.abs(u) ** 3, 90)
    return (16 + 8 * x) * 2.0 ** -23 * (1 + np.minimum(np.abs(u), 4) * 3)
