"""What is measured of the feed-forward operators: the gated projections
act(x Wg^T) * (x Wu^T) with their backward pass, and products of few rows with
4-bit weights that have a scale (and a zero point) for each group.

A 4-bit weight of ``rows`` x ``cols`` with groups of ``group`` columns is held as
  data    uint8 (rows, ld), ld = half a byte a column rounded up to 16 bytes; every
          32-bit word (little endian) holds 8 consecutive columns, column 2 i of
          them in bits 4 i .. 4 i + 3 and column 2 i + 1 in bits 4 i + 16 .. 4 i + 19;
  scales  16-bit (groups, rows), groups = cols / group rounded up, rows of the
          matrix 16-byte aligned;
  zeros   uint8 (groups, rows), rows 16-byte aligned, or none: 8 for all;
and stands for (code - zero) * scale.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    def gated(name, op, M, D, F, act, dtype):
        return {"name": name, "op": op, "M": M, "D": D, "F": F, "act": act, "dtype": dtype}

    def w4(name, op, M, N, K, group, zeros, act, bias, dtype):
        return {"name": name, "op": op, "M": M, "N": N, "K": K, "group": group, "zeros": zeros,
                "act": act, "bias": bias, "dtype": dtype}

    return [
        # the MLP's gated projections for one token: bound by reading the weights
        gated("gated_token", "gated", 1, 4096, 14336, "silu", "bf16"),
        # a decode batch on a large layer
        gated("gated_decode", "gated", 32, 8192, 28672, "silu", "fp16"),
        # a ragged batch on a ragged layer
        gated("gated_ragged", "gated", 1000, 1000, 1000, "gelu", "bf16"),
        # a whole prompt
        gated("gated_prompt", "gated", 8192, 4096, 14336, "silu", "fp16"),
        # forward and backward: a short sequence on a small layer
        gated("train_short", "train", 256, 1024, 4096, "silu", "bf16"),
        # ... ragged
        gated("train_ragged", "train", 1000, 1000, 2000, "gelu", "fp16"),
        # ... a batch of 8192 tokens
        gated("train_batch", "train", 8192, 4096, 14336, "silu", "bf16"),
        # one token through a layer of 4-bit weights
        w4("w4_token", "w4", 1, 14336, 4096, 128, True, "none", False, "fp16"),
        # a decode batch
        w4("w4_decode", "w4", 16, 28672, 8192, 128, False, "none", False, "bf16"),
        # a few rows on a ragged layer, the smallest groups
        w4("w4_ragged", "w4", 5, 1000, 1000, 32, True, "gelu", True, "fp16"),
        # the gated projections with 4-bit weights: one token
        w4("w4_gated_token", "w4_gated", 1, 14336, 4096, 128, True, "silu", False, "bf16"),
        # ... a larger decode batch
        w4("w4_gated_decode", "w4_gated", 64, 14336, 4096, 64, False, "silu", False, "fp16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "train", "w4", "w4_gated"])
    dtype = rng.choice(["fp16", "bf16"])
    if op in ("gated", "train"):
        while True:
            M, D, F = _spread(rng, 1, 8192), _spread(rng, 64, 8192), _spread(rng, 64, 28672)
            if M * D * F <= 8192 * 4096 * 7168 and D * F <= 8192 * 14336:
                return {"op": op, "M": M, "D": D, "F": F,
                        "act": rng.choice(["silu", "silu", "gelu", "relu", "none"]), "dtype": dtype}
    while True:
        N, K = _spread(rng, 64, 28672), _spread(rng, 64, 16384)
        if N * K <= 14336 * 8192:
            return {"op": op, "M": _spread(rng, 1, 64), "N": N, "K": K,
                    "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5,
                    "act": rng.choice(["silu", "gelu"] if op == "w4_gated"
                                      else ["none", "relu", "gelu", "silu"]),
                    "bias": op == "w4" and rng.random() < 0.5, "dtype": dtype}


# ---------------------------------------------------------------------------- inputs ---


def _padded(t, unit=8):
    """A copy whose rows start on 16 bytes, as the library's matrices do."""
    rows, cols = t.shape
    buf = torch.zeros((rows, (cols + unit - 1) // unit * unit), dtype=t.dtype, device=t.device)
    buf[:, :cols] = t
    return buf[:, :cols]


def _activations(g, rows, cols):
    """N(0, 1) with a spread between channels, as activations have."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    return x * torch.exp(0.5 * torch.randn((cols,), generator=g, device="cuda"))


def _weight(g, rows, cols):
    return torch.randn((rows, cols), generator=g, device="cuda") * (1.3 / math.sqrt(cols))


def _quantized(w, group, zeros, dtype):
    """(data, scales, zeros or None) of a weight rounded to the nearest codes."""
    rows, cols = w.shape
    groups = -(-cols // group)
    w = torch.nn.functional.pad(w, (0, groups * group - cols)).view(rows, groups, group)
    if zeros:  # the range from the least to the greatest value
        lo, hi = w.amin(2).clamp_max(0.0), w.amax(2).clamp_min(0.0)
        scale = ((hi - lo) / 15.0).to(dtype)
        zero = torch.round(-lo / scale.float()).clamp(0, 15)
    else:  # a range around 0
        scale = (w.abs().amax(2) / 7.0).to(dtype)
        zero = torch.full((rows, groups), 8.0, device=w.device)
    code = torch.round(w / scale.float()[..., None] + zero[..., None]).clamp(0, 15)
    code = code.to(torch.uint8).view(rows, groups * group)
    size = -(-cols // 32) * 32
    code = torch.nn.functional.pad(code[:, :cols], (0, size - cols)).view(rows, size // 8, 8)
    data = torch.stack((code[..., 0] | code[..., 2] << 4, code[..., 4] | code[..., 6] << 4,
                        code[..., 1] | code[..., 3] << 4, code[..., 5] | code[..., 7] << 4), 2)
    scales = _padded(scale.t().contiguous())
    return data.view(rows, size // 2), scales, \
        _padded(zero.to(torch.uint8).t().contiguous(), 16) if zeros else None


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] in ("gated", "train"):
        M, D, F = case["M"], case["D"], case["F"]
        s["x"] = _padded(_activations(g, M, D).to(dtype))
        s["w_gate"] = _padded(_weight(g, F, D).to(dtype))
        s["w_up"] = _padded(_weight(g, F, D).to(dtype))
        if case["op"] == "train":
            s["dh"] = _padded((0.1 * torch.randn((M, F), generator=g, device="cuda")).to(dtype))
        return s
    M, N, K = case["M"], case["N"], case["K"]
    s["x"] = _padded(_activations(g, M, K).to(dtype))
    for name in ("w", "w_up") if case["op"] == "w4_gated" else ("w",):
        s[name] = _quantized(_weight(g, N, K), case["group"], case["zeros"], dtype)
    s["b"] = (0.5 * torch.randn((N,), generator=g, device="cuda")).to(dtype) if case["bias"] else None
    return s


# ------------------------------------------------------------------------------- run ---


def _act(x, act):
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * torch.erfc(x * -math.sqrt(0.5))
    if act == "relu":
        return torch.clamp_min(x, 0.0)
    return x


def _act_slope(x, act):
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-x))
        return p * (1.0 + x * (1.0 - p))
    if act == "gelu":
        return 0.5 * torch.erfc(x * -math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) * (0.5 / math.pi) ** 0.5
    if act == "relu":
        return (x > 0).to(x.dtype)
    return torch.ones_like(x)


def _dequantized(w, cols, group):
    """The fp32 values of a 4-bit weight."""
    data, scales, zeros = w
    rows = data.shape[0]
    b = data.view(rows, -1, 4)
    code = torch.stack((b[..., 0] & 15, b[..., 2] & 15, b[..., 0] >> 4, b[..., 2] >> 4,
                        b[..., 1] & 15, b[..., 3] & 15, b[..., 1] >> 4, b[..., 3] >> 4), 2)
    code = code.view(rows, -1)[:, :cols].to(torch.float32)
    zero = torch.full_like(scales, 8.0) if zeros is None else zeros
    spread = [v.t().to(torch.float32).repeat_interleave(group, 1)[:, :cols] for v in (zero, scales)]
    return (code - spread[0]) * spread[1]


def run(s):
    op, dtype, act = s["op"], DTYPES[s["dtype"]], s["act"]
    if own:
        import tiled_tensor_core_05_b200 as ttc

        if op == "gated":
            return ttc.gemm_gated(s["x"], s["w_gate"], s["w_up"], act)
        if op == "train":
            h, gate, up = ttc.gemm_gated(s["x"], s["w_gate"], s["w_up"], act, save=True)
            dx, dw_gate, dw_up = ttc.gemm_gated_backward(s["dh"], s["x"], s["w_gate"], s["w_up"],
                                                         gate, up, act)
            return {"h": h, "dx": dx, "dw_gate": dw_gate, "dw_up": dw_up}
        w = ttc.W4Tensor(*s["w"], s["N"], s["K"], s["group"])
        if op == "w4":
            return ttc.gemm_w4(s["x"], w, s["b"], act)
        return ttc.gemm_gated_w4(s["x"], w, ttc.W4Tensor(*s["w_up"], s["N"], s["K"], s["group"]), act)

    x = s["x"].to(torch.float32)
    if op == "w4":
        y = x @ _dequantized(s["w"], s["K"], s["group"]).t()
        if s["b"] is not None:
            y = y + s["b"].to(torch.float32)
        return _act(y, act).to(dtype)
    if op == "w4_gated":
        gate = x @ _dequantized(s["w"], s["K"], s["group"]).t()
        up = x @ _dequantized(s["w_up"], s["K"], s["group"]).t()
        return (_act(gate, act) * up).to(dtype)
    w_gate, w_up = s["w_gate"].to(torch.float32), s["w_up"].to(torch.float32)
    gate, up = x @ w_gate.t(), x @ w_up.t()
    a = _act(gate, act)
    h = (a * up).to(dtype)
    if op == "gated":
        return h
    dh = s["dh"].to(torch.float32)
    d_gate = dh * up * _act_slope(gate, act)
    d_up = dh * a
    return {"h": h, "dx": (d_gate @ w_gate + d_up @ w_up).to(dtype),
            "dw_gate": (d_gate.t() @ x).to(dtype), "dw_up": (d_up.t() @ x).to(dtype)}


# ------------------------------------------------------------------------------ work ---


def work(case):
    M = case["M"]
    if case["op"] in ("gated", "train"):
        D, F = case["D"], case["F"]
        if case["op"] == "gated":
            return {"bytes": 2 * (M * D + 2 * F * D + M * F), "flops": 4 * M * F * D}
        # x, both weights and the gradient of h in; h, the gradients of x and of the weights out
        return {"bytes": 2 * (2 * M * D + 4 * F * D + 2 * M * F), "flops": 12 * M * F * D}
    N, K, groups = case["N"], case["K"], -(-case["K"] // case["group"])
    weight = N * ((K + 1) // 2) + groups * N * (3 if case["zeros"] else 2)
    weights = 2 if case["op"] == "w4_gated" else 1
    return {"bytes": weights * weight + 2 * (M * K + M * N) + (2 * N if case["bias"] else 0),
            "flops": 2 * weights * M * N * K}


# ----------------------------------------------------------------------------- exact ---


def _exact_weight(w, cols, group):
    """The 64-bit values of a 4-bit weight, column by column of each word."""
    data, scales, zeros = w
    words = data.contiguous().view(torch.int32)
    v = torch.empty((data.shape[0], cols), dtype=torch.float64, device=data.device)
    for j in range(8):
        at = 4 * (j // 2) + 16 * (j % 2)
        n = (cols - j + 7) // 8
        v[:, j::8] = ((words >> at) & 15)[:, :n].double()
    for i in range(scales.shape[0]):
        part = v[:, i * group:(i + 1) * group]
        part -= 8.0 if zeros is None else zeros[i].double()[:, None]
        part *= scales[i].double()[:, None]
    return v


def _exact_act(x, act):
    """(value, derivative)"""
    if act == "silu":
        p = torch.sigmoid(x)
        return x * p, p + x * p * torch.sigmoid(-x)
    if act == "gelu":
        p = torch.special.ndtr(x)
        return x * p, p + x * torch.exp(x.square() / -2) / math.sqrt(2 * math.pi)
    if act == "relu":
        return x.clamp(min=0), torch.heaviside(x, torch.zeros((), dtype=x.dtype, device=x.device))
    return x, x.new_ones(())


def exact(case, seed):
    s = prepare(case, seed)
    x, act = s["x"].double(), case["act"]
    if case["op"] == "w4":
        y = torch.matmul(x, _exact_weight(s["w"], case["K"], case["group"]).t())
        if s["b"] is not None:
            y += s["b"].double()
        return _exact_act(y, act)[0]
    if case["op"] == "w4_gated":
        gate = torch.matmul(x, _exact_weight(s["w"], case["K"], case["group"]).t())
        up = torch.matmul(x, _exact_weight(s["w_up"], case["K"], case["group"]).t())
        return _exact_act(gate, act)[0].mul_(up)
    wg, wu = s["w_gate"].double(), s["w_up"].double()
    a, slope = _exact_act(torch.matmul(x, wg.t()), act)
    up = torch.matmul(x, wu.t())
    h = a * up
    if case["op"] == "gated":
        return h
    dh = s["dh"].double()
    d_up = a.mul_(dh)
    d_gate = up.mul_(slope).mul_(dh)
    return {"h": h, "dx": torch.addmm(torch.matmul(d_gate, wg), d_up, wu),
            "dw_gate": torch.matmul(d_gate.t(), x), "dw_up": torch.matmul(d_up.t(), x)}
