"""Plain definitions, in numpy with 64-bit arithmetic, of the RMS norm with an
8-bit output and of MXFP8 operands whose rows lie in groups."""
import numpy as np

import fp4_reference as ref4

E4M3, E5M2 = 0, 1
EMAX = {E4M3: 8, E5M2: 15}


def e5m2_byte(v):
    """Byte of an E5M2 value (finite, representable)."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    e = np.maximum(np.frexp(a)[1] - 1, -14)
    m = a / np.ldexp(1.0, e - 2)                      # 0..7
    code = np.where(m >= 4, (e + 15) * 4 + (m - 4), m)
    return (code + 128 * np.signbit(v)).astype(np.uint8)


def e5m2_value(b):
    b = np.asarray(b, np.uint8).astype(np.int64)
    e, m = (b >> 2) & 31, b & 3
    v = np.where(e > 0, np.ldexp(1.0 + m / 4, e - 15), np.ldexp(m / 4.0, -14))
    v = np.where((b & 127) > 124, np.nan, np.where((b & 127) == 124, np.inf, v))
    return np.where(b & 128, -v, v)


def value(b, fmt):
    return ref4.e4m3_value(b) if fmt == E4M3 else e5m2_value(b)


def mx_rows(x, fmt):
    """x [R, C] -> (bytes [R, C], scale codes [R, ceil(C / 32)])."""
    R, C = x.shape
    t = np.zeros((R, -(-C // 32) * 32))
    t[:, :C] = x
    t = t.reshape(R, -1, 32)
    top = np.abs(t).max(axis=2, initial=0.0)
    bad = ~np.isfinite(top)
    top = np.where(bad, 1.0, top)
    code = np.where(top == 0, 0, np.clip(np.frexp(top)[1] - 1 - EMAX[fmt] + 127, 0, 254))
    with np.errstate(invalid="ignore"):
        v = np.where(bad[..., None], 0.0, t) * np.ldexp(1.0, 127 - code)[..., None]
    if fmt == E4M3:
        b = ref4.e4m3_byte(ref4.round_float(v, 3, -6, 448.0))
    else:
        b = e5m2_byte(ref4.round_float(v, 2, -14, 57344.0))
    b = np.where(bad[..., None], 0x7F, b)
    return b.reshape(R, -1)[:, :C].astype(np.uint8), np.where(bad, 0xFF, code).astype(np.uint8)


def mx_values(b, code, fmt):
    s = np.ldexp(1.0, code.astype(np.int64) - 127)
    s[code == 0xFF] = np.nan
    return value(b, fmt) * np.repeat(s, 32, axis=1)[:, :b.shape[1]]


def place(atoms, code, row0, block0, per_row):
    """Writes scale codes [R, B] of rows row0 on and blocks block0 on into atoms
    (flat bytes, `per_row` atoms to a 128-row block)."""
    r = row0 + np.arange(code.shape[0])[:, None]
    b = block0 + np.arange(code.shape[1])[None, :]
    atoms[((r // 128) * per_row + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = code


def take(atoms, R, B, row0, block0, per_row):
    r = row0 + np.arange(R)[:, None]
    b = block0 + np.arange(B)[None, :]
    return atoms[((r // 128) * per_row + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4]


class Groups:
    """Where the groups of an operand lie."""

    def __init__(self, ends, equal=False):
        self.ends, self.E = list(ends), len(ends) - 1
        if equal:
            n = ends[-1] // self.E
            self.first = [e * -(-n // 128) for e in range(self.E)]
        else:
            self.first = [a // 128 + e for e, a in enumerate(ends[:-1])]

    def __iter__(self):
        for e in range(self.E):
            yield e, self.ends[e], self.ends[e + 1], self.first[e]


def cast(x, groups, fmt, store, rows=True, cols=True):
    """Casts rows x [S, C] in groups into store's arrays (q, q_scales flat, q_t,
    qt_scales flat), leaving everything that no group owns."""
    C = x.shape[1]
    kb = -(-C // 128)
    for _, a, z, b in groups:
        n = -(-(z - a) // 128)
        if rows and z > a:
            q, code = mx_rows(x[a:z], fmt)
            store["q"][a:z] = q
            whole = np.zeros((128 * n, 4 * kb), np.uint8)
            whole[:z - a, :code.shape[1]] = code
            place(store["q_scales"], whole, 128 * b, 0, kb)
        if cols and z > a:
            t = np.zeros((C, 128 * n))
            t[:, :z - a] = x[a:z].T
            q, code = mx_rows(t, fmt)
            store["q_t"][:, 128 * b:128 * (b + n)] = q
            whole = np.zeros((128 * kb, 4 * n), np.uint8)
            whole[:C] = code
            place(store["qt_scales"], whole, 0, 4 * b, store["q_t"].shape[1] // 128)


def group_rows(store, groups, fmt):
    """Values of every group's rows [n, C], from the row orientation."""
    C = store["q"].shape[1]
    kb = -(-C // 128)
    for _, a, z, b in groups:
        yield mx_values(store["q"][a:z], take(store["q_scales"], z - a, -(-C // 32), 128 * b, 0, kb), fmt)


def group_cols(store, groups, fmt):
    """Values of every group's columns [C, n], from the transposed orientation."""
    C, width = store["q_t"].shape
    for _, a, z, b in groups:
        n = -(-(z - a) // 32)
        code = take(store["qt_scales"], C, n, 0, 4 * b, width // 128)
        yield mx_values(store["q_t"][:, 128 * b:128 * b + z - a], code, fmt)


# ---------------------------------------------------------------- the norm

U32 = 2.0 ** -24       # half a step of fp32, relative


def chain(C):
    """Most roundings that one term of a sum over a row meets: the terms of a
    thread (up to 32 held, C / 512 in long rows) one after the other, five
    steps in a warp, up to 16 warps."""
    return 32 + C / 512 + 5 + 16


def rstd_error(C):
    """Relative error of rstd: the sum's (of terms of one sign), a division and
    an addition, halved by the root, and the root's own."""
    return (0.5 * (chain(C) + 2) + 1) * U32


def norm(h, w, eps):
    rstd = 1.0 / np.sqrt((h ** 2).sum(axis=1) / h.shape[1] + eps)
    return rstd, h * rstd[:, None] * w


def norm_scales(y, row):
    T, C = y.shape
    n = C if row else 128
    t = np.zeros((T, -(-C // n) * n))
    t[:, :C] = np.abs(y)
    return np.maximum(t.reshape(T, -1, n).max(axis=2) / 448.0, 1e-12)     # [T, tiles]


def norm_backward(dy, h, w, rstd, dres):
    """(dx, dw, bound on dx's error, bound on dw's) without their last rounding."""
    T, C = h.shape
    r = rstd[:, None]
    n, g = h * r, dy * w
    mean = (g * n).mean(axis=1, keepdims=True)
    dx = r * (g - n * mean) + dres
    # each of g, n is off by a rounding, their products' sum by one for every
    # step of the chain, and a handful more follow
    size = np.abs(g * n).mean(axis=1, keepdims=True)
    dx_err = r * (np.abs(g) + np.abs(n) * size) * (chain(C) + 8) * U32 + np.abs(dx) * U32
    dw = (dy * n).sum(axis=0)
    dw_err = np.abs(dy * n).sum(axis=0) * (T + 64) * U32   # rows, warps, blocks one after the other
    return dx, dw, dx_err, dw_err
