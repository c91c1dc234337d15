"""Cases that measure the norm and the experts' operators in 8 bits.

Five operators in six forms: the root-mean-square norm with the residual's addition and an
E4M3 output under scales ("norm"), its backward pass ("norm_backward"), the
MXFP8 cast of routed rows ("cast"), and the three products of a linear layer
per expert: forward ("fprop"), the gradient of its input ("dgrad") and of its
weights ("wgrad").  With ``own`` false every operator is computed in elementary
torch operations in fp32; with ``own`` true through this repository's entry
points.  ``exact`` restates each definition in 64 bits.

Rows of a matrix lie in groups, one after the other: group e holds rows
offsets[e] to offsets[e + 1], and rows behind the last offset are nobody's.
MXFP8 has one E8M0 scale, 2^(floor(log2 amax) - 8) for E4M3 or - 15 for E5M2,
per 32 elements: along a row, or down a column from the group's first row on.
Scale bytes lie in atoms of 128 rows x 128 elements (512 bytes): the scale of
row r, block b is byte (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4 of atom
(r / 128, b / 4).  A group starts at 128-row block offsets[e] / 128 + e of the
row scales, and at 128 times that column of the transposed bytes; equal groups
(weights) of n rows start at e * ceil(n / 128).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E4M3, E5M2 = "e4m3", "e5m2"
FLOAT8 = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
TOP = {E4M3: 448.0, E5M2: 57344.0}
EMAX = {E4M3: 8, E5M2: 15}
EPS = 1e-6

# The transformer layer of this repository's benchmark: 15872 tokens, hidden
# size 4096; an 8192 x 4096 activation in its quantize benchmark.
TOKENS, HIDDEN = 15872, 4096
# A generic layer of experts: half the hidden size inside, two experts a token.
EXPERTS, INNER = 32, 2048


def listed():
    return [
        # the norm in front of a linear over the layer's whole token batch, in training
        dict(name="norm tile batch", op="norm", T=TOKENS, C=HIDDEN, dtype="bf16", w_dtype="bf16", add=True, y=True,
             scaling="tile"),
        # the same in front of one decoded token's products, which want the 8-bit row alone
        dict(name="norm row one token", op="norm", T=1, C=HIDDEN, dtype="bf16", w_dtype="bf16", add=True, y=False,
             scaling="row"),
        # an odd-sized layer in fp32, no residual
        dict(name="norm tile ragged", op="norm", T=1003, C=2570, dtype="fp32", w_dtype="fp32", add=False, y=True,
             scaling="tile"),
        # its backward pass, joined by the residual's gradient
        dict(name="norm backward batch", op="norm_backward", T=8192, C=HIDDEN, dtype="bf16", w_dtype="bf16", add=True),
        dict(name="norm backward ragged", op="norm_backward", T=333, C=1111, dtype="fp32", w_dtype="fp32", add=False),
        # 8192 tokens to two experts each, both orientations, as a training step needs them
        dict(name="cast batch", op="cast", tokens=8192, top=2, E=EXPERTS, spare=0, C=HIDDEN, dtype="bf16", fmt=E4M3,
             both=True),
        # a small decoding batch in front of many experts
        dict(name="cast 13 tokens", op="cast", tokens=13, top=4, E=64, spare=12, C=2000, dtype="fp32", fmt=E4M3,
             both=False),
        # the experts' up projection of that batch
        dict(name="fprop batch", op="fprop", tokens=8192, top=2, E=EXPERTS, spare=0, N=INNER, K=HIDDEN, out="bf16"),
        # one decoded token through eight of 64 experts: their weights are what is read
        dict(name="fprop one token", op="fprop", tokens=1, top=8, E=64, spare=0, N=INNER, K=HIDDEN, out="bf16"),
        # the gradient of a small odd-sized layer's input, gradients in E5M2, fp32 result
        dict(name="dgrad ragged", op="dgrad", tokens=501, top=2, E=12, spare=22, N=1008, K=2000, out="fp32"),
        # the weights' gradient of the up projection
        dict(name="wgrad batch", op="wgrad", tokens=8192, top=2, E=EXPERTS, spare=0, N=INNER, K=HIDDEN, out="bf16"),
        # that of a small layer, some of whose experts get few rows or none, fp32 result
        dict(name="wgrad ragged", op="wgrad", tokens=259, top=3, E=12, spare=5, N=336, K=656, out="fp32"),
    ]


def _size(rng, low, high):
    return max(low, min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "cast", "cast", "fprop", "fprop", "dgrad", "wgrad", "wgrad"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    while True:
        if op in ("norm", "norm_backward"):
            case = dict(op=op, T=_size(rng, 1, TOKENS), C=_size(rng, 16, 16384), dtype=dtype,
                        w_dtype=rng.choice(["bf16", "fp32"]), add=rng.random() < 0.6)
            if op == "norm":
                case.update(y=rng.random() < 0.7, scaling=rng.choice(["tile", "row"]))
            fits = case["T"] * case["C"] * (2 if dtype == "fp32" else 1) <= 8192 * HIDDEN
        else:
            E = _size(rng, 1, 128)
            case = dict(op=op, tokens=_size(rng, 1, 8192), top=rng.randint(1, min(8, E)), E=E,
                        spare=rng.choice([0, rng.randint(1, 300)]))
            S = case["tokens"] * case["top"]
            if op == "cast":
                case.update(C=16 * _size(rng, 1, 512), dtype=dtype, fmt=rng.choice([E4M3, E4M3, E5M2]),
                            both=rng.random() < 0.6)
                fits = S * case["C"] <= 16384 * HIDDEN // 2
            else:
                case.update(N=16 * _size(rng, 1, 512), K=16 * _size(rng, 2, 512), out=rng.choice(["bf16", "fp32"]))
                NK = case["N"] * case["K"]
                fits = E * NK <= 16 * INNER * HIDDEN and S * NK <= 8192 * INNER * HIDDEN
        if fits:
            return case


# ------------------------------------------------------- plain form, in fp32

_POWERS = {}


def _power(e, dtype=torch.float32):
    """2^e of whole numbers from -160 to 160, every one exact (torch's own power and ldexp are not on every device)."""
    if dtype not in _POWERS:
        _POWERS[dtype] = torch.tensor([2.0 ** k for k in range(-160, 161)], dtype=torch.float64).to(e.device, dtype)
    return _POWERS[dtype][e.long() + 160]


def _over(x, d):
    """x / d as a division of tensors (by a Python number torch multiplies with its reciprocal)."""
    return x / torch.full((), d, dtype=x.dtype, device=x.device)


def _amax_scale(top):
    return torch.clamp(_over(top, 448.0), min=1e-12)


def _tiles(x, n=128):
    """[R, C] -> [R, ceil(C / n), n], zeros past C."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % n)).view(x.shape[0], -1, n)


def _mx(x, fmt):
    """x [R, C] -> (bytes [R, C], scale codes [R, ceil(C / 32)])."""
    t = _tiles(x.float(), 32)
    top = t.abs().amax(dim=2)
    code = torch.clamp(torch.frexp(top)[1] - 1 - EMAX[fmt] + 127, 0, 254)
    code = torch.where(top == 0, 0, code)
    q = torch.clamp(t * _power(127 - code)[..., None], -TOP[fmt], TOP[fmt]).to(FLOAT8[fmt])
    return q.view(torch.uint8).view(x.shape[0], -1)[:, :x.shape[1]], code.to(torch.uint8)


def _atoms(code):
    """Codes [R, b] -> atoms [ceil(R / 128), ceil(b / 4), 512], zeros past the matrix."""
    c = torch.nn.functional.pad(code, (0, -code.shape[1] % 4, 0, -code.shape[0] % 128))
    return c.view(c.shape[0] // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).reshape(c.shape[0] // 128, -1, 512)


def _codes(atoms):
    """Atoms [rb, kb, 512] -> codes [128 rb, 4 kb]."""
    rb, kb = atoms.shape[:2]
    return atoms.view(rb, kb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(128 * rb, 4 * kb)


def _starts(ends, equal=0):
    """First 128-row block of every group, and the number of blocks there are."""
    if equal:
        per = (equal + 127) // 128
        return [e * per for e in range(len(ends) - 1)], (len(ends) - 1) * per
    return [a // 128 + e for e, a in enumerate(ends[:-1])], None


def _blocks(S, E):
    return S // 128 + E


def _cast(x, ends, fmt, store, rows, cols, equal=0):
    """Writes what is asked for of x [S, C], whose groups end at `ends`, into `store`."""
    C = x.shape[1]
    for e, b in enumerate(_starts(ends, equal)[0]):
        a, z = ends[e], ends[e + 1]
        n = (z - a + 127) // 128
        if n == 0:
            continue
        if rows:
            store["q"][a:z], code = _mx(x[a:z], fmt)
            store["q_scales"][b:b + n] = _atoms(code)
        if cols:
            q, code = _mx(torch.nn.functional.pad(x[a:z], (0, 0, 0, a - z + 128 * n)).t(), fmt)
            store["q_t"][:, 128 * b:128 * (b + n)] = q
            store["qt_scales"][:, b:b + n] = _atoms(code)
    return store


def _storage(S, C, blocks, rows, cols):
    new = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device="cuda")
    kb = (C + 127) // 128
    got = dict(q=new(S, C), q_scales=new(blocks, kb, 512)) if rows else {}
    if cols:
        got.update(q_t=new(C, 128 * blocks), qt_scales=new(kb, blocks, 512))
    return got


def _values(q, code, fmt):
    """What bytes [R, K] under scale codes [>= R, >= K / 32] stand for, in fp32."""
    s = _power(code[:q.shape[0]].int() - 127).repeat_interleave(32, dim=1)
    return q.contiguous().view(FLOAT8[fmt]).float() * s[:, :q.shape[1]]


def _group_rows(op, e, ends, fmt, equal=0):
    """Group e's rows of an operand, from the row orientation."""
    b, n = _starts(ends, equal)[0][e], (ends[e + 1] - ends[e] + 127) // 128
    return _values(op["q"][ends[e]:ends[e + 1]], _codes(op["q_scales"][b:b + n]), fmt)


def _group_cols(op, e, ends, fmt, equal=0):
    """Group e's columns of the transposed orientation, [C, rows of the group]."""
    b, n = _starts(ends, equal)[0][e], (ends[e + 1] - ends[e] + 127) // 128
    return _values(op["q_t"][:, 128 * b:128 * b + ends[e + 1] - ends[e]], _codes(op["qt_scales"][:, b:b + n]), fmt)


# ------------------------------------------------------------------- inputs

def _route(case, r):
    """A router's choice: (token of every grouped row, offsets), experts of unlike favour."""
    T, E, top = case["tokens"], case["E"], case["top"]
    score = torch.randn((T, E), generator=r, device="cuda") + torch.randn((E,), generator=r, device="cuda")
    expert = score.topk(top, dim=1).indices.reshape(-1)
    order = torch.sort(expert, stable=True).indices
    ends = torch.cumsum(torch.bincount(expert, minlength=E), 0)
    return (order // top).int(), torch.cat((ends.new_zeros(1), ends)).int()


def _inputs(case, seed):
    """The drawn numbers of a case, before anything is laid out."""
    r = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, scale=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=r, device="cuda") * scale).to(dtype)

    op = case["op"]
    if op in ("norm", "norm_backward"):
        dt, T, C = DTYPES[case["dtype"]], case["T"], case["C"]
        got = dict(x=normal(T, C, scale=2.0, dtype=dt),
                   w=(1.0 + 0.2 * torch.randn((C,), generator=r, device="cuda")).to(DTYPES[case["w_dtype"]]))
        if case["add"]:
            got["residual"] = normal(T, C, dtype=dt)
        if op == "norm_backward":
            got["dy"] = normal(T, C, scale=1e-2, dtype=dt)
        return got
    index, offsets = _route(case, r)
    S = index.shape[0]
    got = dict(index=index, offsets=offsets)
    if op == "cast":
        got["x"] = normal(case["tokens"], case["C"], dtype=DTYPES[case["dtype"]])
        return got
    if op in ("fprop", "wgrad"):
        got["x"] = normal(S, case["K"])
    if op in ("dgrad", "wgrad"):
        got["g"] = normal(S, case["N"], scale=1e-3)
    if op != "wgrad":
        got["w"] = normal(case["E"] * case["N"], case["K"], scale=0.02)
    return got


def _rstd(x):
    return torch.rsqrt((x.float() * x.float()).mean(dim=1) + EPS)


def prepare(case, seed):
    state, op = dict(case, **_inputs(case, seed)), case["op"]
    if op == "norm_backward":
        state["h"] = state.pop("x")
        state["rstd"] = _rstd(state["h"])
    if op in ("norm", "norm_backward"):
        return state
    E, S = case["E"], state["index"].shape[0] + case["spare"]
    ends = state["ends"] = state["offsets"].tolist()
    state["S"] = S
    if op == "cast":
        pad = torch.full((case["spare"],), -1, dtype=torch.int32, device="cuda")  # rows behind the last group
        state["index"] = torch.cat((state["index"], pad))
        state["store"] = _storage(S, case["C"], _blocks(S, E), True, case["both"])
        return state
    del state["index"]
    N, K, out = case["N"], case["K"], DTYPES[case["out"]]
    if op in ("fprop", "wgrad"):
        x = state.pop("x")
        state["x_op"] = _cast(x, ends, E4M3, _storage(S, K, _blocks(S, E), op == "fprop", op == "wgrad"),
                              op == "fprop", op == "wgrad")
    if op in ("dgrad", "wgrad"):
        g = state.pop("g")
        state["g_op"] = _cast(g, ends, E5M2, _storage(S, N, _blocks(S, E), op == "dgrad", op == "wgrad"),
                              op == "dgrad", op == "wgrad")
    if op == "wgrad":
        return state
    operand = state["x_op"] if op == "fprop" else state["g_op"]
    operand["q"][ends[-1]:] = 0x7F  # nobody's rows hold whatever was there: NaN
    w, equal = state.pop("w"), [N * e for e in range(E + 1)]
    state["w_op"] = _cast(w, equal, E4M3, _storage(E * N, K, E * ((N + 127) // 128), op == "fprop", op == "dgrad"),
                          op == "fprop", op == "dgrad", equal=N)
    state["result"] = torch.zeros((S, N if op == "fprop" else K), dtype=out, device="cuda")
    return state


# ---------------------------------------------------------------------- run

def run(state):
    return (_run_own if own else _run_plain)(state)


def _shown(store, fmt):
    """Bytes as the values they stand for, scales as the codes that they are."""
    return {k: v.view(FLOAT8[fmt]) if k in ("q", "q_t") else v.view(-1) for k, v in store.items()}


def _run_plain(s):
    op = s["op"]
    if op == "norm":
        dt, h, got = DTYPES[s["dtype"]], s["x"], {}
        if s["add"]:
            h = got["h"] = (s["x"].float() + s["residual"].float()).to(dt)
        got["rstd"] = _rstd(h)
        y = h.float() * got["rstd"][:, None] * s["w"].float()
        t = _tiles(y) if s["scaling"] == "tile" else y[:, None]
        scale = _amax_scale(t.abs().amax(dim=2))
        q = (t / scale[..., None]).to(torch.float8_e4m3fn).view(y.shape[0], -1)[:, :y.shape[1]]
        if s["y"]:
            got["y"] = y.to(dt)
        return dict(got, q=q.contiguous(), scales=scale.t().contiguous())
    if op == "norm_backward":
        dt, h, dy = DTYPES[s["dtype"]], s["h"].float(), s["dy"].float()
        xh, g = h * s["rstd"][:, None], dy * s["w"].float()
        dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(dim=1, keepdim=True))
        if s["add"]:
            dx = dx + s["residual"].float()
        return dict(dx=dx.to(dt), dw=(dy * xh).sum(dim=0).to(s["w"].dtype))
    ends = s["ends"]
    if op == "cast":
        rows = s["x"].float()[s["index"][:ends[-1]].long()]
        return _shown(_cast(rows, ends, s["fmt"], s["store"], True, s["both"]), s["fmt"])
    E, N, K, out = s["E"], s["N"], s["K"], DTYPES[s["out"]]
    if op == "wgrad":
        dw = torch.empty((E, N, K), dtype=out, device="cuda")
        for e in range(E):
            dw[e] = (_group_cols(s["g_op"], e, ends, E5M2) @ _group_cols(s["x_op"], e, ends, E4M3).t()).to(out)
        return dw
    equal = [N * e for e in range(E + 1)]
    for e in range(E):
        if ends[e + 1] > ends[e]:
            if op == "fprop":
                y = _group_rows(s["x_op"], e, ends, E4M3) @ _group_rows(s["w_op"], e, equal, E4M3, N).t()
            else:
                y = _group_rows(s["g_op"], e, ends, E5M2) @ _group_cols(s["w_op"], e, equal, E4M3, N).t()
            s["result"][ends[e]:ends[e + 1]] = y.to(out)
    return s["result"]


def _run_own(s):
    import scaled_quantize_fp8_warp_gb300 as fq
    op = s["op"]
    if op == "norm":
        got = fq.fp8_rmsnorm(s["x"], s["w"], residual=s.get("residual"), eps=EPS,
                             scaling=fq.SCALE_TILE_1x128 if s["scaling"] == "tile" else fq.SCALE_ROW, want_y=s["y"])
        out = dict(rstd=got.rstd, q=got.q.view(torch.float8_e4m3fn), scales=got.scales.view(-1, s["T"]))
        if s["add"]:
            out["h"] = got.h
        if s["y"]:
            out["y"] = got.y
        return out
    if op == "norm_backward":
        dx, dw = fq.fp8_rmsnorm_backward(s["dy"], s["h"], s["w"], s["rstd"],
                                         dresidual=s.get("residual"))
        return dict(dx=dx, dw=dw)
    E = s["E"]

    def operand(rows, cols, groups, fmt, offsets, st):
        return fq.ExpertsOperand(rows, cols, groups, fq.E4M3 if fmt == E4M3 else fq.E5M2, offsets, st.get("q"),
                                 st.get("q_scales"), st.get("q_t"), st.get("qt_scales"))

    if op == "cast":
        store = operand(s["S"], s["C"], E, s["fmt"], s["offsets"], s["store"])
        fq.fp8_quantize_experts(s["x"], E, offsets=s["offsets"], index=s["index"], cols=s["both"], fmt=store.fmt,
                                out=store)
        return _shown(s["store"], s["fmt"])
    N, K, out = s["N"], s["K"], DTYPES[s["out"]]
    if op in ("fprop", "wgrad"):
        x = operand(s["S"], K, E, E4M3, s["offsets"], s["x_op"])
    if op in ("dgrad", "wgrad"):
        g = operand(s["S"], N, E, E5M2, s["offsets"], s["g_op"])
    if op == "wgrad":
        return fq.fp8_experts_wgrad(g, x, out_dtype=out)
    w = operand(E * N, K, E, E4M3, None, s["w_op"])
    if op == "fprop":
        return fq.fp8_experts_fprop(x, w, out=s["result"])
    return fq.fp8_experts_dgrad(g, w, out=s["result"])


def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        n, size = case["T"] * case["C"], 2 if case["dtype"] == "bf16" else 4
        if op == "norm":
            scales = case["T"] * 4 * ((case["C"] + 127) // 128 if case["scaling"] == "tile" else 1)
            return dict(bytes=n * (size * (1 + 2 * case["add"] + case["y"]) + 1) + scales, flops=0)
        return dict(bytes=n * size * (3 + case["add"]), flops=0)
    S, E = case["tokens"] * case["top"], case["E"]
    if op == "cast":
        read = case["tokens"] * case["C"] * (2 if case["dtype"] == "bf16" else 4)
        return dict(bytes=read + S * case["C"] * 33 / 32 * (2 if case["both"] else 1), flops=0)
    N, K, size = case["N"], case["K"], 2 if case["out"] == "bf16" else 4
    met = E * (1.0 - (1.0 - case["top"] / E) ** case["tokens"])  # experts with a row, for a fair router
    if op == "wgrad":
        return dict(bytes=S * (N + K) * 33 / 32 + E * N * K * size, flops=2 * S * N * K)
    contract, result = (K, N) if op == "fprop" else (N, K)
    return dict(bytes=(S * contract + met * N * K) * 33 / 32 + S * result * size, flops=2 * S * N * K)


# -------------------------------------------- the definitions again, in 64 bits

def _round_to(v, bits, lowest, top):
    """v rounded to nearest even with `bits` fraction bits, exponents from `lowest` up, clipped to +-top."""
    e = torch.clamp(torch.frexp(v)[1] - 1, min=lowest)
    step = _power(e - bits, torch.float64)
    return torch.clamp(torch.round(v / step) * step, -top, top)


def _exact_mx(x, fmt):
    """x [R, C] in float64 -> (the 8-bit values before their scale [R, C], exponents [R, ceil(C / 32)])."""
    R, C = x.shape
    t = torch.zeros(R, -(-C // 32) * 32, dtype=torch.float64, device=x.device)
    t[:, :C] = x
    t = t.reshape(R, -1, 32)
    top = t.abs().max(dim=2).values
    e = torch.clamp(torch.floor(torch.log2(top)) - EMAX[fmt], min=-127.0)
    v = t / _power(e, torch.float64)[..., None]
    v = _round_to(v, 3, -6, 448.0) if fmt == E4M3 else _round_to(v, 2, -14, 57344.0)
    return v.reshape(R, -1)[:, :C], e


def _exact_values(x, fmt):
    v, e = _exact_mx(x, fmt)
    return v * _power(e, torch.float64).repeat_interleave(32, dim=1)[:, :x.shape[1]]


def _place(codes, e, row0, block0, per_row):
    """codes.view(-1)[byte of (row, block)] = e + 127, rows from row0 on and blocks from block0 on."""
    r = torch.arange(e.shape[0], device=e.device)[:, None] + row0
    b = torch.arange(e.shape[1], device=e.device)[None, :] + block0
    at = ((r // 128) * per_row + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
    codes[at.reshape(-1)] = (e + 127).to(torch.uint8).reshape(-1)


def exact(case, seed):
    op = case["op"]
    x = _inputs(case, seed)
    if op == "norm":
        dt, h = DTYPES[case["dtype"]], x["x"].double()
        got = {}
        if case["add"]:
            got["h"] = (h + x["residual"].double()).to(dt).double()  # it is kept in the input's type
            h = got["h"]
        rstd = 1.0 / torch.sqrt((h ** 2).sum(dim=1) / case["C"] + EPS)
        y = h * rstd[:, None] * x["w"].double()
        n = 128 if case["scaling"] == "tile" else case["C"]
        t = torch.zeros(case["T"], -(-case["C"] // n) * n, dtype=torch.float64, device=y.device)
        t[:, :case["C"]] = y
        t = t.reshape(case["T"], -1, n)
        s = torch.clamp(t.abs().max(dim=2).values / 448, min=1e-12).float().double()  # held in 32 bits
        q = _round_to(t / s[..., None], 3, -6, 448.0).reshape(case["T"], -1)[:, :case["C"]]
        if case["y"]:
            got["y"] = y
        return dict(got, rstd=rstd, q=q, scales=s.t())
    if op == "norm_backward":
        h, dy, w = (x[k].double() for k in ("x", "dy", "w"))
        rstd = _rstd(x["x"]).double()[:, None]  # an input, held in 32 bits
        inner = (dy * w * h).sum(dim=1, keepdim=True) * rstd ** 2 / case["C"]
        dx = rstd * (dy * w - h * inner) + (x["residual"].double() if case["add"] else 0.0)
        return dict(dx=dx, dw=(dy * h * rstd).sum(dim=0))
    ends, E = x["offsets"].tolist(), case["E"]
    S = ends[-1] + case["spare"]
    if op == "cast":
        C, blocks, kb = case["C"], S // 128 + E, (case["C"] + 127) // 128
        got = dict(q=torch.zeros(S, C, dtype=torch.float64, device="cuda"),
                   q_scales=torch.zeros(blocks * kb * 512, dtype=torch.uint8, device="cuda"))
        if case["both"]:
            got.update(q_t=torch.zeros(C, 128 * blocks, dtype=torch.float64, device="cuda"),
                       qt_scales=torch.zeros(blocks * kb * 512, dtype=torch.uint8, device="cuda"))
        for e in range(E):
            a, z, first = ends[e], ends[e + 1], 128 * (ends[e] // 128 + e)
            if a == z:
                continue
            t = x["x"][x["index"][a:z].long()].double()
            got["q"][a:z], power = _exact_mx(t, case["fmt"])
            _place(got["q_scales"], power, first, 0, kb)
            if case["both"]:
                got["q_t"][:, first:first + z - a], power = _exact_mx(t.t(), case["fmt"])
                _place(got["qt_scales"], power, 0, first // 32, blocks)
        return got
    N, K = case["N"], case["K"]
    if op == "wgrad":
        dw = torch.zeros((E, N, K), dtype=torch.float64, device="cuda")
        for e in range(E):
            g, t = (x[k][ends[e]:ends[e + 1]].double().t() for k in ("g", "x"))
            if g.shape[1]:
                dw[e] = _exact_values(g, E5M2) @ _exact_values(t, E4M3).t()
        return dw
    result = torch.zeros((S, N if op == "fprop" else K), dtype=torch.float64, device="cuda")
    for e in range(E):
        a, z, w = ends[e], ends[e + 1], x["w"][N * e:N * (e + 1)].double()
        if a == z:
            continue
        if op == "fprop":
            result[a:z] = _exact_values(x["x"][a:z].double(), E4M3) @ _exact_values(w, E4M3).t()
        else:
            result[a:z] = _exact_values(x["g"][a:z].double(), E5M2) @ _exact_values(w.t(), E4M3).t()
    return result
