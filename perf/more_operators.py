"""The operators around microscaled 8- and 4-bit matrices, as a serving step calls them.

Four operators, each with a plain form in elementary torch operations:

* ``quant``  bf16 rows quantised to a microscaled format, and read back to bf16.
* ``norm``   residual addition and RMS norm, quantised to 8 bits, and read back.
* ``lin``    y = x W^T of two microscaled matrices.
* ``mlp``    silu(x W_gate^T) * (x W_up^T) of microscaled matrices, to bf16 or
             quantised to 8 bits and read back.

A matrix [rows, cols] is held as codes and scales, one scale for ``group``
neighbouring elements of a row; a value is code * scale * g, g a power of two
for the whole matrix.

* ``nvfp4``  e2m1 codes, e4m3 scales for 16 elements
* ``mxfp4``  e2m1 codes, power-of-two (e8m0) scales for 32 elements, g = 1
* ``mxfp8``  e4m3 codes, power-of-two (e8m0) scales for 32 elements, g = 1

Codes lie row by row (4-bit ones two to a byte, the even element low).  Scales
lie in tiles of 128 rows x 4 groups, 512 bytes each, a row of tiles after the
other; ``_scale_places`` gives the byte of (row, group).
"""

import math

import torch

own = False

GROUP = {"nvfp4": 16, "mxfp4": 32, "mxfp8": 32}
TOP = {"nvfp4": 6.0, "mxfp4": 6.0, "mxfp8": 448.0}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the input of a 70B layer's gate_up, one decode step of 128 sequences
        {"name": "norm_decode_128", "op": "norm", "m": 128, "k": 8192, "res": True},
        # the same of a prompt of 8 x 4096 tokens
        {"name": "norm_prefill_32768", "op": "norm", "m": 32768, "k": 8192, "res": True},
        # an odd number of rows, an odd number of groups, a first layer (no residual yet)
        {"name": "norm_odd_1021", "op": "norm", "m": 1021, "k": 1376, "res": False},
        # the input of an 8B layer's down projection in a decode step of 64 sequences
        {"name": "quant_decode_64", "op": "quant", "fmt": "mxfp8", "m": 64, "k": 14336, "pad": 0},
        # the 70B layer's gate_up weight, quantised when a checkpoint is loaded
        {"name": "quant_weight_70b", "op": "quant", "fmt": "nvfp4", "m": 57344, "k": 8192, "pad": 0},
        # columns of a wider matrix, odd rows and groups
        {"name": "quant_columns_1021", "op": "quant", "fmt": "mxfp4", "m": 1021, "k": 2080, "pad": 1032},
        # the smallest product: one sequence's o_proj of an 8B layer
        {"name": "lin_one_8b", "op": "lin", "fmt": "nvfp4", "m": 1, "n": 4096, "k": 4096},
        # the 70B down projection of 128 decode sequences: 28672 inputs
        {"name": "lin_decode_70b", "op": "lin", "fmt": "nvfp4", "m": 128, "n": 8192, "k": 28672},
        # an odd chunk through odd sizes
        {"name": "lin_odd_421", "op": "lin", "fmt": "mxfp4", "m": 421, "n": 1384, "k": 2080},
        # the 70B o_proj of a prompt of 8 x 4096 tokens
        {"name": "lin_prefill_70b", "op": "lin", "fmt": "mxfp8", "m": 32768, "n": 8192, "k": 8192},
        # the 8B gate_up of 64 decode sequences, handed on in 8 bits
        {"name": "mlp_decode_8b", "op": "mlp", "fmt": "mxfp8", "m": 64, "n": 14336, "k": 4096, "out": "mxfp8"},
        # the 70B gate_up of 32 decode sequences beside two prompt chunks of 2048 tokens
        {"name": "mlp_mixed_70b", "op": "mlp", "fmt": "nvfp4", "m": 4128, "n": 28672, "k": 8192, "out": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    return max(1, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step))) * step


def draw(rng):
    op, fmt = rng.choice(["norm", "quant", "lin", "lin", "mlp"]), rng.choice(["nvfp4", "mxfp4", "mxfp8"])
    if op == "norm":
        return {"op": op, "m": _log(rng, 1, 16384), "k": _log(rng, 64, 16384, 32), "res": rng.random() < 0.75}
    if op == "quant":
        return {"op": op, "fmt": fmt, "m": _log(rng, 1, 16384), "k": _log(rng, 32, 28672, 32),
                "pad": rng.choice([0, 0, 8, 1032])}
    out = rng.choice(["bf16", "mxfp8"])
    m, k = _log(rng, 1, 8192), _log(rng, 32, 28672, 32)
    n = _log(rng, 32, 28672, 32 if op == "mlp" and out == "mxfp8" else 8)
    while m * n * k > 5e11:
        m = m // 2
    return {"op": op, "fmt": fmt, "m": m, "n": n, "k": k, **({"out": out} if op == "mlp" else {})}


def _bytes(fmt, rows, cols):
    """A matrix's codes and scales (scales of the rows and groups that are there)."""
    return rows * (cols if fmt == "mxfp8" else cols // 2) + rows * (cols // GROUP[fmt])


def work(c):
    m, k, n = c["m"], c["k"], c.get("n", 0)
    if c["op"] == "quant":  # read, write; read again, write what it holds
        return {"bytes": 4 * m * k + 2 * _bytes(c["fmt"], m, k), "flops": 6 * m * k}
    if c["op"] == "norm":
        return {"bytes": (8 if c["res"] else 6) * m * k + 2 * k + 2 * _bytes("mxfp8", m, k), "flops": 11 * m * k}
    if c["op"] == "lin":
        return {"bytes": _bytes(c["fmt"], m, k) + _bytes(c["fmt"], n, k) + 2 * m * n, "flops": 2 * m * n * k}
    byte = _bytes(c["fmt"], m, k) + 2 * _bytes(c["fmt"], n, k) + 2 * m * n
    return {"bytes": byte + (2 * _bytes("mxfp8", m, n) if c["out"] == "mxfp8" else 0), "flops": 4 * m * n * k}


# ---------------------------------------------------------------------------
# the formats
# ---------------------------------------------------------------------------
def _scale_places(rows, groups, dev):
    """[rows, groups] bytes of the scales."""
    r, s = torch.arange(rows, device=dev)[:, None], torch.arange(groups, device=dev)
    return ((r // 128) * (-(-groups // 4)) + s // 4) * 512 + (r % 32) * 16 + r % 128 // 32 * 4 + s % 4


def _scale_bytes(fmt, rows, cols):
    return -(-rows // 128) * -(-(cols // GROUP[fmt]) // 4) * 512


def _quantise(x, fmt, g):
    """x [rows, cols] fp32 -> (values of the codes [rows, cols], scales [rows, groups]), fp32.

    nvfp4: scale e4m3(amax / (6 g)).  mxfp4, mxfp8: the smallest power of two
    with which no element is beyond the largest code.  Codes to nearest, ties to
    even.  Exact for bf16 inputs: their quotients are on a border of the codes or
    2^-8 away from it."""
    y = (x / g).view(x.shape[0], -1, GROUP[fmt])
    amax = y.abs().amax(-1)
    if fmt == "nvfp4":
        s = (amax / 6).clamp(max=448.0).to(torch.float8_e4m3fn).float()
        y = torch.where(s[..., None] > 0, y / torch.where(s > 0, s, 1.0)[..., None], 0.0)
    else:
        mant, top = math.frexp(TOP[fmt])
        f = torch.frexp(amax)
        e = torch.where(amax > 0, f.exponent - top + (f.mantissa > mant), -127).clamp(-127, 127)
        s = torch.ldexp(torch.ones_like(amax), e)
        y = torch.ldexp(y, -e[..., None])
    if fmt == "mxfp8":
        q = y.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    else:
        a = y.abs()
        code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() \
            + (a >= 3.5).byte() + (a > 5.0).byte()
        q = torch.tensor(GRID, device=x.device)[code.int()] * torch.sign(y)
    return q.view(x.shape), s


def _read(codes, scales, fmt, cols, g):
    """[rows, cols] fp32 values of a matrix."""
    rows, groups = codes.shape[0], cols // GROUP[fmt]
    s = scales[_scale_places(rows, groups, codes.device)]
    if fmt == "nvfp4":
        s = s.view(torch.float8_e4m3fn).float()
    else:
        s = torch.ldexp(torch.ones(s.shape, device=codes.device), s.int() - 127)
    if fmt == "mxfp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        grid = torch.tensor(GRID + tuple(-x for x in GRID), device=codes.device)
        v = grid[torch.stack([codes & 15, codes >> 4], -1).view(rows, cols).int()]
    return (v.view(rows, groups, -1) * (s * g)[..., None]).view(rows, cols)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(g, m, k):
    """Activations: a few channels far larger than the others."""
    return _normal(g, m, k) * (1.0 + 15.0 * (torch.rand(k, generator=g, device="cuda") > 0.99))


def _stored(fmt, rows, cols, dev="cuda"):
    """An empty matrix: (codes, scales)."""
    return (torch.empty(rows, cols if fmt == "mxfp8" else cols // 2, dtype=torch.uint8, device=dev),
            torch.zeros(_scale_bytes(fmt, rows, cols), dtype=torch.uint8, device=dev))


def _pack(x, fmt, g):
    """x [rows, cols] as a stored matrix, for the inputs."""
    rows, cols = x.shape
    codes, scales = _stored(fmt, rows, cols)
    for r in range(0, rows, 8192):  # by parts: the large weights
        q, s = _quantise(x[r:r + 8192].float(), fmt, g)
        at = _scale_places(rows, cols // GROUP[fmt], x.device)[r:r + 8192]
        scales[at] = s.to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "nvfp4" else \
            (torch.frexp(s).exponent + 126).byte()
        if fmt == "mxfp8":
            codes[r:r + 8192] = q.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            a = q.abs()
            c = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).byte() + 8 * torch.signbit(q).byte()
            codes[r:r + 8192] = c[:, 0::2] | (c[:, 1::2] << 4)
    return codes, scales


def _matrix(x, fmt, g):
    g = g if fmt == "nvfp4" else 1.0
    codes, scales = _pack(x, fmt, g)
    return {"fmt": fmt, "cols": x.shape[1], "codes": codes, "scales": scales, "g": g}


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 6151 + 29)
    m, k = c["m"], c["k"]
    st = {"op": c["op"], "c": c}
    if c["op"] == "quant":
        wide = (_rows(g, m, k + c["pad"])).bfloat16()
        st["x"] = wide[:, :k]
        st["g"] = 2.0 ** -5 if c["fmt"] == "nvfp4" else 1.0
        st["out"] = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
        st["to"] = {"fmt": c["fmt"], "cols": k, "g": st["g"], **dict(zip(("codes", "scales"), _stored(c["fmt"], m, k)))}
    elif c["op"] == "norm":
        st["x"], st["eps"] = _rows(g, m, k).bfloat16(), 1e-5
        st["res"] = _rows(g, m, k).bfloat16() if c["res"] else None
        st["gamma"] = (1 + 0.2 * _normal(g, k)).bfloat16()
        st["res_out"] = torch.empty_like(st["x"])
        st["out"] = torch.empty_like(st["x"])
        st["to"] = {"fmt": "mxfp8", "cols": k, "g": 1.0, **dict(zip(("codes", "scales"), _stored("mxfp8", m, k)))}
    else:
        n = c["n"]
        st["xq"] = _matrix(_rows(g, m, k), c["fmt"], 2.0 ** -5)
        st["w"] = [_matrix(_normal(g, n, k).mul_(k ** -0.5), c["fmt"], 2.0 ** -13)
                   for _ in range(2 if c["op"] == "mlp" else 1)]
        st["out"] = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        if c.get("out") == "mxfp8":
            st["to"] = {"fmt": "mxfp8", "cols": n, "g": 1.0, **dict(zip(("codes", "scales"), _stored("mxfp8", m, n)))}
    if own:
        from llama_decoder_layer_gb300 import binding as lb
        kinds = {"nvfp4": lb.LLAMA_MX_NVFP4, "mxfp4": lb.LLAMA_MX_FP4, "mxfp8": lb.LLAMA_MX_FP8}

        def handle(d):
            return lb.MxMatrix(kinds[d["fmt"]], d["cols"], d["codes"], d["scales"], d["g"])

        st["to_h"] = handle(st["to"]) if "to" in st else None
        if "xq" in st:
            st["x_h"], st["w_h"] = handle(st["xq"]), [handle(w) for w in st["w"]]
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(st):
    if own:
        return _run_own(st)
    c = st["c"]
    if c["op"] == "quant":
        q, s = _quantise(st["x"].float(), c["fmt"], st["g"])
        return _values(q, s, c["fmt"], st["g"]).bfloat16()
    if c["op"] == "norm":
        r = st["x"].float() if st["res"] is None else st["x"].float() + st["res"].float()
        r = r.bfloat16()
        h = r.float()
        h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + st["eps"]) * st["gamma"].float()
        return _values(*_quantise(h, "mxfp8", 1.0), "mxfp8", 1.0).bfloat16(), r
    x = _read(st["xq"]["codes"], st["xq"]["scales"], c["fmt"], c["k"], st["xq"]["g"])
    y = [x @ _read(w["codes"], w["scales"], c["fmt"], c["k"], w["g"]).T for w in st["w"]]
    if c["op"] == "lin":
        return y[0].bfloat16()
    a = y[0] / (1 + torch.exp(-y[0])) * y[1]
    return a.bfloat16() if c["out"] == "bf16" else _values(*_quantise(a, "mxfp8", 1.0), "mxfp8", 1.0).bfloat16()


def _values(q, s, fmt, g):
    return (q.view(*s.shape, GROUP[fmt]) * (s * g)[..., None]).view(q.shape)


def _run_own(st):
    from llama_decoder_layer_gb300 import binding as lb
    op = st["op"]
    if op == "lin":
        lb.linear_mx(st["x_h"], st["w_h"][0], st["out"])
        return st["out"]
    if op == "mlp":
        to = st["out"] if st["to_h"] is None else st["to_h"]
        lb.gate_up_silu_mx(st["x_h"], st["w_h"][0], st["w_h"][1], to)
        if st["to_h"] is not None:
            lb.dequantize_mx(st["to_h"], st["out"])
        return st["out"]
    if op == "quant":
        lb.quantize_mx(st["x"], st["to_h"])
        lb.dequantize_mx(st["to_h"], st["out"])
        return st["out"]
    lb.fused_add_rmsnorm_mx(st["x"], st["res"], st["res_out"], st["to_h"], st["gamma"], st["eps"])
    lb.dequantize_mx(st["to_h"], st["out"])
    return st["out"], st["res_out"]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _nearest(a, bits, low, top):
    """a >= 0 to the nearest of a float with `bits` significant bits and a least exponent `low`, ties to even."""
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** low)))
    e = e + (torch.exp2(e + 1) <= a).double() - (torch.exp2(e) > a.clamp(min=2.0 ** low)).double()
    step = torch.exp2(e - (bits - 1))
    return (torch.round(a / step) * step).clamp(max=top)


def _exact_values(x, fmt, g):
    """What x [rows, cols] in 64 bits is once stored."""
    b = x.reshape(-1, GROUP[fmt]) / g
    amax = b.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        s = _nearest(amax / 6, 4, -6, 448.0)
    else:
        e = torch.ceil(torch.log2((amax / TOP[fmt]).clamp(min=2.0 ** -127)))
        e = e - (amax <= TOP[fmt] * torch.exp2(e - 1)).double() + (amax > TOP[fmt] * torch.exp2(e)).double()
        s = torch.exp2(e.clamp(-127, 127))
    a = torch.where(s > 0, b.abs() / torch.where(s > 0, s, 1.0), 0.0)
    v = _nearest(a, 4, -6, 448.0) if fmt == "mxfp8" else _nearest(a, 2, 0, 6.0)
    return (torch.copysign(v, b) * s * g).reshape(x.shape)


def _exact_read(d):
    """The values of a stored matrix, from the bits of the format."""
    codes, cols, grp = d["codes"].long(), d["cols"], GROUP[d["fmt"]]
    rows, tiles = codes.shape[0], -(-(cols // grp) // 4)
    raw = d["scales"].view(-1, tiles, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, tiles * 4)[:rows, :cols // grp].long()
    if d["fmt"] == "nvfp4":
        s = torch.where(raw >= 8, (1 + (raw & 7) / 8.0) * torch.exp2((raw >> 3).double() - 7), (raw & 7) / 512.0)
    else:
        s = torch.exp2(raw.double() - 127)
    if d["fmt"] == "mxfp8":
        e, f = (codes >> 3) & 15, (codes & 7) / 8.0
        v = torch.where(e > 0, (1 + f) * torch.exp2(e.double() - 7), f * 2.0 ** -6)
        v = torch.where(codes >= 128, -v, v)
    else:
        nib = torch.empty(rows, cols, dtype=torch.long, device=codes.device)
        nib[:, 0::2], nib[:, 1::2] = codes & 15, codes >> 4
        e, f = (nib >> 1) & 3, (nib & 1) * 0.5
        v = torch.where(e > 0, (1 + f) * torch.exp2(e.double() - 1), f)
        v = torch.where(nib >= 8, -v, v)
    return v.double() * s.repeat_interleave(grp, 1) * d["g"]


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "quant":
        return torch.cat([_exact_values(x.double(), c["fmt"], st["g"]) for x in st["x"].split(8192)])
    if c["op"] == "norm":
        outs, sums = [], []
        for i, x in enumerate(st["x"].split(8192)):
            r = x.double()
            if c["res"]:
                r = (r + st["res"].split(8192)[i].double()).bfloat16().double()
            sums.append(r)
            h = r / (r.square().sum(-1, keepdim=True) / c["k"] + st["eps"]).sqrt() * st["gamma"].double()
            outs.append(_exact_values(h, "mxfp8", 1.0))
        return torch.cat(outs), torch.cat(sums)
    x = _exact_read(st["xq"])
    ys = []
    for w in st["w"]:
        part = [dict(w, codes=w["codes"][r:r + 8192], scales=w["scales"].view(-(-c["n"] // 128), -1)[r // 128:].reshape(-1))
                for r in range(0, c["n"], 8192)]
        ys.append(torch.cat([torch.einsum("mk,nk->mn", x, _exact_read(p)) for p in part], 1))
    if c["op"] == "lin":
        return ys[0]
    a = ys[0] * torch.sigmoid(ys[0]) * ys[1]
    return a if c["out"] == "bf16" else _exact_values(a, "mxfp8", 1.0)
