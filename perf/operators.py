"""What is measured of the microscaled (MX) operators: quantisation, the RMS
norm that produces MX activations, and the product of two MX matrices.

Formats are those of the OCP Microscaling Formats (MX) specification v1.0:
blocks of 32 elements along a row share one E8M0 scale; the elements are E4M3
("mxfp8") or E2M1 ("mxfp4", two to a byte, the even one in the low half).

A matrix of ``rows`` x ``cols`` is held as
  data    uint8 (rows, ld), ld = the bytes of a row rounded up to 16;
  scales  uint8, flat: for each 128 rows and each 4 blocks a tile of 512 bytes,
          the scale of row r and block b at byte (r % 32) * 16 +
          (r % 128 // 32) * 4 + b % 4 of tile (r // 128) * ceil(cols / 128) + b // 4;
          places without a block hold 0.
"""
import math

import torch

own = False

BLOCK = 32
EMAX = {"mxfp8": 8, "mxfp4": 2}      # exponent of the format's largest power of two
LARGEST = {"mxfp8": 448.0, "mxfp4": 6.0}
MIN_EXP = {"mxfp8": -6, "mxfp4": 0}  # smallest normal exponent
MANT = {"mxfp8": 3, "mxfp4": 1}      # mantissa bits
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-6


def listed():
    def norm(name, rows, cols, residual, fmt, dtype):
        return {"name": name, "op": "norm", "rows": rows, "cols": cols, "residual": residual,
                "format": fmt, "dtype": dtype}

    def quantize(name, rows, cols, fmt, dtype):
        return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "format": fmt,
                "dtype": dtype}

    def product(name, M, N, K, fmt, act, bias, dtype):
        return {"name": name, "op": "product", "M": M, "N": N, "K": K, "format": fmt, "act": act,
                "bias": bias, "dtype": dtype}

    return [
        # one token before an MLP: the residual stream is updated and normed straight to 8 bits
        norm("norm_token", 1, 4096, True, "mxfp8", "fp16"),
        # a whole prompt before the MLP up-projection
        norm("norm_prompt", 8192, 4096, True, "mxfp8", "fp16"),
        # a final norm whose reader wants 16 bits, no residual, ragged rows
        norm("norm_ragged", 1000, 1000, False, "none", "bf16"),
        # activations of a decode batch, 4 bits
        quantize("quantize_decode", 32, 8192, "mxfp4", "fp16"),
        # a layer's weight, quantised when a model is loaded
        quantize("quantize_weight", 14336, 4096, "mxfp4", "bf16"),
        # activations after an activation function, 8 bits
        quantize("quantize_prompt", 8192, 14336, "mxfp8", "fp16"),
        # single token and decode batch: bound by reading the weight
        product("product_token", 1, 14336, 4096, "mxfp8", "none", False, "fp16"),
        product("product_decode", 32, 28672, 8192, "mxfp4", "relu", False, "fp16"),
        # a middling batch on a ragged layer
        product("product_ragged", 1000, 1000, 1000, "mxfp4", "none", True, "bf16"),
        # a short prompt: too few tiles to fill the card
        product("product_short", 256, 4096, 8192, "mxfp8", "none", False, "bf16"),
        # the MLP up-projection of a prompt with its bias and GELU
        product("product_mlp_up", 8192, 14336, 4096, "mxfp4", "gelu", True, "fp16"),
        # the large cube in 8 bits
        product("product_cube", 8192, 8192, 8192, "mxfp8", "relu", False, "fp16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "product", "product"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "norm":
        cols = _spread(rng, 32, 16384)
        rows = _spread(rng, 1, min(16384, 8192 * 4096 // cols))
        return {"op": op, "rows": rows, "cols": cols, "residual": rng.random() < 0.5,
                "format": rng.choice(["none", "mxfp8", "mxfp8", "mxfp4"]), "dtype": dtype}
    if op == "quantize":
        cols = _spread(rng, 32, 16384)
        rows = _spread(rng, 1, min(28672, 8192 * 14336 // cols))
        return {"op": op, "rows": rows, "cols": cols, "format": rng.choice(["mxfp4", "mxfp8"]),
                "dtype": dtype}
    while True:
        M, N, K = _spread(rng, 1, 8192), _spread(rng, 64, 28672), _spread(rng, 64, 16384)
        if M * N * K <= 8192 * 8192 * 4096 and N * K <= 28672 * 8192:
            return {"op": op, "M": M, "N": N, "K": K, "format": rng.choice(["mxfp4", "mxfp8"]),
                    "act": rng.choice(["none", "relu", "gelu"]), "bias": rng.random() < 0.5,
                    "dtype": dtype}


# ------------------------------------------------------------ the layout of MX data ---


def _row_bytes(cols, fmt):
    return cols if fmt == "mxfp8" else (cols + 1) // 2


def _tile_scales(s):
    """(rows, blocks) scale bytes -> the flat tiled layout."""
    rows, nb = s.shape
    R, B = -(-rows // 128), -(-nb // 4)
    t = torch.zeros((R * 128, B * 4), dtype=s.dtype, device=s.device)
    t[:rows, :nb] = s
    return t.view(R, 4, 32, B, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile_scales(flat, rows, cols):
    R, B = -(-rows // 128), -(-cols // 128)
    t = flat.view(R, B, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R * 128, B * 4)
    return t[:rows, :-(-cols // BLOCK)]


def _pack(q, fmt):
    """Element values (rows, cols) -> data bytes (rows, ld)."""
    rows, cols = q.shape
    n = _row_bytes(cols, fmt)
    data = torch.zeros((rows, (n + 15) // 16 * 16), dtype=torch.uint8, device=q.device)
    if fmt == "mxfp8":
        data[:, :cols] = q.to(torch.float8_e4m3fn).view(torch.uint8)
        return data
    mag = q.abs()
    code = torch.zeros(q.shape, dtype=torch.uint8, device=q.device)
    for v in E2M1[1:]:
        code += (mag >= v).to(torch.uint8)
    code += torch.signbit(q).to(torch.uint8) * 8
    if cols % 2:
        code = torch.nn.functional.pad(code, (0, 1))
    data[:, :n] = code[:, 0::2] + code[:, 1::2] * 16
    return data


def _quantize(x, fmt):
    """(element values, scale bytes (rows, blocks)) of the rows of x, in x's type (32 or 64 bits)."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    if cols % BLOCK:
        x = torch.nn.functional.pad(x, (0, nb * BLOCK - cols))
    x = x.view(rows, nb, BLOCK)
    amax = x.abs().amax(2)
    exp = torch.frexp(amax)[1] - 1 - EMAX[fmt]  # floor(log2(amax)) - emax
    exp = torch.where(amax > 0, exp.clamp(-127, 127), torch.full_like(exp, -127))
    y = torch.ldexp(x, -exp[..., None])
    e = (torch.frexp(y)[1] - 1).clamp_min(MIN_EXP[fmt]) - MANT[fmt]
    q = torch.ldexp(torch.round(torch.ldexp(y, -e)), e)  # round() takes ties to even
    q = torch.where(torch.signbit(x), -q.abs(), q.abs()).clamp(-LARGEST[fmt], LARGEST[fmt])
    return q.view(rows, nb * BLOCK)[:, :cols], (exp + 127).to(torch.uint8)


def _scaled(q, s):
    """Element values and scale bytes (rows, blocks) -> what they stand for."""
    cols = q.shape[1]
    x = torch.ldexp(torch.ones((), dtype=q.dtype, device=q.device), s.to(torch.int32) - 127)
    return q * x.repeat_interleave(BLOCK, 1)[:, :cols]


def _dequantize(data, scales, rows, cols, fmt):
    """The fp32 values of an MX matrix."""
    n = _row_bytes(cols, fmt)
    if fmt == "mxfp8":
        q = data[:, :n].view(torch.float8_e4m3fn).to(torch.float32)
    else:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=data.device)
        c = data[:, :n].to(torch.int32)
        q = torch.stack((table[c & 15], table[c >> 4]), 2).view(rows, 2 * n)[:, :cols]
    return _scaled(q, _untile_scales(scales, rows, cols))


# ---------------------------------------------------------------------------- inputs ---


def _padded(t):
    """A copy whose rows start on 16 bytes, as the library's matrices do."""
    rows, cols = t.shape
    buf = torch.empty((rows, (cols + 7) // 8 * 8), dtype=t.dtype, device=t.device)
    buf[:, :cols] = t
    return buf[:, :cols]


def _activations(g, rows, cols):
    """N(0, 1) with a spread between channels, as activations have."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    return x * torch.exp(0.5 * torch.randn((cols,), generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = dict(case)
    if op == "norm":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _padded(_activations(g, rows, cols).to(dtype))
        s["r"] = _padded(_activations(g, rows, cols).to(dtype)) if case["residual"] else None
        s["w"] = (1.0 + 0.2 * torch.randn((cols,), generator=g, device="cuda")).to(dtype)
    elif op == "quantize":
        s["x"] = _padded(_activations(g, case["rows"], case["cols"]).to(dtype))
    else:
        M, N, K, fmt = case["M"], case["N"], case["K"], case["format"]
        for name, rows in (("a", M), ("b", N)):
            if name == "a":
                v = _activations(g, rows, K)
            else:
                v = 0.02 * torch.randn((rows, K), generator=g, device="cuda")
            q, e = _quantize(v, fmt)
            s[name] = (_pack(q, fmt), _tile_scales(e))
            del v, q, e
        s["bias"] = None
        if case["bias"]:
            s["bias"] = (0.5 * torch.randn((N,), generator=g, device="cuda")).to(dtype)
    return s


# ------------------------------------------------------------------------------- run ---


def _as_values(data, scales, rows, cols, fmt, values):
    """How MX outputs are returned: 8-bit elements and scales as views of the bytes, 4-bit ones as
    the values that they stand for."""
    out = {"scales": scales.view(torch.float8_e8m0fnu)}
    if fmt == "mxfp8":
        out["elements"] = data[:, :cols].view(torch.float8_e4m3fn)
    else:
        out["values"] = values
    return out


def run(s):
    op, fmt, dtype = s["op"], s["format"], DTYPES[s["dtype"]]
    if own:
        import tiled_tensor_core_05_b200 as ttc

        def as_values(q):
            values = ttc.mx_dequantize(q, dtype=dtype) if fmt == "mxfp4" else None
            return _as_values(q.data, q.scales, q.rows, q.cols, fmt, values)

        if op == "product":
            a = ttc.MxTensor(*s["a"], s["M"], s["K"], fmt)
            b = ttc.MxTensor(*s["b"], s["N"], s["K"], fmt)
            return ttc.gemm_mx(a, b, s["bias"], s["act"], dtype=dtype)
        if op == "quantize":
            return as_values(ttc.mx_quantize(s["x"], fmt))
        y = ttc.rms_norm(s["x"], s["w"], EPS, residual=s["r"],
                         format=None if fmt == "none" else fmt)
        y, h = y if s["residual"] else (y, None)
        out = {"y": y} if fmt == "none" else as_values(y)
        if h is not None:
            out["h"] = h
        return out

    def as_values(q, e):
        return _as_values(_pack(q, fmt) if fmt == "mxfp8" else None, _tile_scales(e), *q.shape, fmt,
                          _scaled(q, e).to(dtype) if fmt == "mxfp4" else None)

    if op == "product":
        a = _dequantize(*s["a"], s["M"], s["K"], fmt)
        b = _dequantize(*s["b"], s["N"], s["K"], fmt)
        c = a @ b.t()
        if s["bias"] is not None:
            c = c + s["bias"].to(torch.float32)
        if s["act"] == "relu":
            c = torch.clamp_min(c, 0.0)
        elif s["act"] == "gelu":
            c = 0.5 * c * torch.erfc(c * -math.sqrt(0.5))
        return c.to(dtype)
    if op == "quantize":
        return as_values(*_quantize(s["x"].to(torch.float32), fmt))
    h = s["x"].to(torch.float32)
    out = {}
    if s["residual"]:
        out["h"] = (h + s["r"].to(torch.float32)).to(dtype)
        h = out["h"].to(torch.float32)
    if fmt != "none":
        h = h.to(torch.float64)  # which element a value becomes is decided next to a border
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["w"].to(h.dtype)
    if fmt == "none":
        out["y"] = y.to(dtype)
    else:
        out.update(as_values(*_quantize(y, fmt)))
    return out


# ------------------------------------------------------------------------------ work ---


def _mx_bytes(rows, cols, fmt):
    return rows * (_row_bytes(cols, fmt) + -(-cols // BLOCK))


def work(case):
    op, fmt = case["op"], case["format"]
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        size = _mx_bytes(M, K, fmt) + _mx_bytes(N, K, fmt) + 2 * M * N + (2 * N if case["bias"] else 0)
        return {"bytes": size, "flops": 2 * M * N * K}
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    size = 2 * n if fmt == "none" else _mx_bytes(rows, cols, fmt)
    if fmt == "mxfp4":  # read again, and the values written
        size += size + 2 * n
    if op == "quantize":
        return {"bytes": size + 2 * n, "flops": 2 * n}
    return {"bytes": size + 2 * n + 2 * cols + (4 * n if case["residual"] else 0), "flops": 4 * n}


# ----------------------------------------------------------------------------- exact ---


def _magnitudes(fmt):
    """All non-negative finite values of the element type, by code."""
    bits = MANT[fmt]
    got = []
    for code in range(8 if fmt == "mxfp4" else 127):
        e, m = code >> bits, code & ((1 << bits) - 1)
        bias = 1 - MIN_EXP[fmt]
        got.append((m / 2 ** bits) * 2.0 ** MIN_EXP[fmt] if e == 0
                   else (1 + m / 2 ** bits) * 2.0 ** (e - bias))
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def _exact_quantize(x, fmt):
    """(values of the elements, scale exponents (rows, blocks)) from the definition: the nearest
    element by search among all of them, ties to the even code."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    full = torch.zeros((rows, nb * BLOCK), dtype=torch.float64, device=x.device)
    full[:, :cols] = x
    full = full.view(rows * nb, BLOCK)
    amax = full.abs().max(1).values
    powers = torch.tensor([2.0 ** k for k in range(-170, 129)], dtype=torch.float64, device=x.device)
    exp = torch.bucketize(amax, powers, right=True) - 171 - EMAX[fmt]
    exp = exp.clamp(-127, 127)
    y = full.abs() / torch.exp2(exp.to(torch.float64))[:, None]
    table = _magnitudes(fmt)
    mids = (table[1:] + table[:-1]) / 2
    low, high = torch.bucketize(y, mids), torch.bucketize(y, mids, right=True)
    code = torch.where(low % 2 == 0, low, high)
    q = torch.copysign(table[code], full)
    return q.view(rows, nb * BLOCK)[:, :cols], exp.view(rows, nb)


def _exact_values(data, scales, rows, cols, fmt):
    """The 64-bit values of an MX matrix, bit by bit."""
    r = torch.arange(rows, device=data.device)[:, None]
    b = torch.arange(-(-cols // BLOCK), device=data.device)[None, :]
    at = ((r // 128) * -(-cols // 128) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
    exp = scales[at].to(torch.float64) - 127
    k = torch.arange(cols, device=data.device)
    code = data[:, :cols] if fmt == "mxfp8" else (data[:, k // 2] >> (4 * (k % 2)).to(torch.uint8)) & 15
    sign = 128 if fmt == "mxfp8" else 8
    v = _magnitudes(fmt)[(code & (sign - 1)).to(torch.int64)]
    v = torch.where(code >= sign, -v, v)
    x = torch.exp2(exp)
    for j in range(0, cols, BLOCK):
        v[:, j:j + BLOCK] *= x[:, j // BLOCK, None]
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt = case["op"], case["format"]
    if op == "product":
        a = _exact_values(*s["a"], s["M"], s["K"], fmt)
        c = torch.matmul(a, _exact_values(*s["b"], s["N"], s["K"], fmt).t())
        if s["bias"] is not None:
            c += s["bias"].double()
        if s["act"] == "relu":
            c = c.clamp(min=0)
        elif s["act"] == "gelu":
            c = c * torch.special.ndtr(c)
        return c

    def mx(y):
        q, e = _exact_quantize(y, fmt)
        x = torch.exp2(e.to(torch.float64))
        padded = torch.full((-(-y.shape[0] // 128) * 128, -(-y.shape[1] // 128) * 4), 2.0 ** -127,
                            dtype=torch.float64, device=y.device)
        padded[:x.shape[0], :x.shape[1]] = x
        tiles = padded.reshape(-1, 4, 32, padded.shape[1] // 4, 4).permute(0, 3, 2, 1, 4)
        out = {"scales": tiles.reshape(-1)}
        if fmt == "mxfp8":
            out["elements"] = q
        else:
            out["values"] = q * torch.repeat_interleave(x, BLOCK, dim=1)[:, :y.shape[1]]
        return out

    if op == "quantize":
        return mx(s["x"].double())
    h, out = s["x"].double(), {}
    if case["residual"]:
        out["h"] = h + s["r"].double()
        h = out["h"].to(s["x"].dtype).double()  # the norm reads the stream as it is stored
    y = h / torch.sqrt(h.square().sum(1, keepdim=True) / case["cols"] + EPS) * s["w"].double()
    if fmt == "none":
        out["y"] = y
    else:
        out.update(mx(y))
    return out
