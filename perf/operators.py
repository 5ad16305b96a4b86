"""Cases for the narrow-format MLP operators: MXFP4 quantization and product, and the
SwiGLU and RMSNorm that keep their activations in 8 bits for the backward pass.

A case's "op" names the operator:

  quantize   x -> E2M1 codes with one E8M0 scale per 32 columns -> the values they stand for
  transpose  the same down the rows, codes written transposed, from a raw tensor or from an 8-bit checkpoint
  gemm       C = A B^T, B in E2M1, A in E2M1, E4M3 or E5M2, all with one E8M0 scale per 32 of K
  swiglu     h = silu(g) u as E4M3 codes, (g, u) kept as E4M3 codes; the gradient from the kept codes
  rmsnorm    y = x / rms(x) w as E4M3 codes, x kept as E4M3 codes; the gradients from the kept codes

`run` is one pass: with `own` false in elementary torch operations, with `own` true by the
library's calls.  Codes are returned as the values they stand for.
"""
import torch

own = False

# (mantissa bits, smallest normal exponent, largest finite value) of each element format
FORMATS = {"e2m1": (1, 0, 6.0), "e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
EPS = 1e-6


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # the 7B-class MLP weight, quantized again after each optimizer step
        {"name": "quantize-weight-7b", "op": "quantize", "rows": 18944, "cols": 3584, "dtype": "bf16", "rule": "floor"},
        # one token's hidden state on its way into a 4-bit product: latency
        {"name": "quantize-token", "op": "quantize", "rows": 1, "cols": 3584, "dtype": "bf16", "rule": "ceil"},
        # the 1.5B-class weight from its fp32 master copy, for the data gradient's product
        {"name": "transpose-weight-1p5b", "op": "transpose", "rows": 8960, "cols": 1536, "source": "f32", "to": "e2m1",
         "rule": "floor"},
        # a linear layer's kept input, turned for its weight gradient; a token count that fills no tile
        {"name": "transpose-kept-odd", "op": "transpose", "rows": 4099, "cols": 8960, "source": "e4m3", "to": "e4m3",
         "rule": "ceil"},
        # decoding: one token against the 7B-class up projection
        {"name": "gemm-token-7b", "op": "gemm", "m": 1, "n": 18944, "k": 3584, "a": "e4m3"},
        # a small ragged batch of decoded tokens, both sides in 4 bits
        {"name": "gemm-batch-odd", "op": "gemm", "m": 37, "n": 1536, "k": 8960, "a": "e2m1"},
        # training and prefill: the 7B-class up projection with both sides in 4 bits
        {"name": "gemm-4bit-7b", "op": "gemm", "m": 8192, "n": 18944, "k": 3584, "a": "e2m1"},
        # the data gradient: 8-bit gradients times the 4-bit transposed weight
        {"name": "gemm-dgrad-7b", "op": "gemm", "m": 8192, "n": 3584, "k": 18944, "a": "e5m2"},
        # a training step's activation, forward and backward, at the 7B-class width
        {"name": "swiglu-train-7b", "op": "swiglu", "rows": 8192, "cols": 18944, "dtype": "bf16", "pass": "train"},
        # serving a small batch: forward only, nothing kept
        {"name": "swiglu-serve-odd", "op": "swiglu", "rows": 37, "cols": 8960, "dtype": "bf16", "pass": "serve"},
        # a training step's norm, forward and backward
        {"name": "rmsnorm-train-7b", "op": "rmsnorm", "rows": 16384, "cols": 3584, "dtype": "bf16", "pass": "train"},
        # one token's norm: latency
        {"name": "rmsnorm-token", "op": "rmsnorm", "rows": 1, "cols": 1536, "dtype": "f32", "pass": "serve"},
    ]


def draw(rng):
    def spread(low, high):
        return int(round(low * (high / low) ** rng.random()))

    def width(low, high, step):
        return max(low, spread(low, high) // step * step)

    op = rng.choice(("quantize", "transpose", "gemm", "gemm", "swiglu", "rmsnorm"))
    if op == "quantize":
        return {"op": op, "rows": spread(1, 16384), "cols": width(32, 4096, 32), "dtype": rng.choice(("f32", "bf16")),
                "rule": rng.choice(("floor", "ceil"))}
    if op == "transpose":
        return {"op": op, "rows": spread(1, 8192), "cols": width(32, 4096, 32),
                "source": rng.choice(("f32", "bf16", "e4m3", "e5m2")), "to": rng.choice(("e2m1", "e4m3", "e5m2")),
                "rule": rng.choice(("floor", "ceil"))}
    if op == "gemm":
        return {"op": op, "m": spread(1, 8192), "n": spread(16, 16384), "k": width(128, 3584, 128),
                "a": rng.choice(("e2m1", "e4m3", "e5m2"))}
    case = {"op": op, "rows": spread(1, 8192), "cols": width(32, 16384 if op == "swiglu" else 8192, 32),
            "dtype": rng.choice(("f32", "bf16")), "pass": rng.choice(("train", "train", "serve"))}
    if op == "swiglu" and case["dtype"] == "f32":
        case["rows"] = max(1, case["rows"] // 2)
    return case


def padded(rows):
    return (rows + 127) // 128 * 128


def work(case):
    op = case["op"]
    code = {"e2m1": 0.5, "e4m3": 1.0, "e5m2": 1.0}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (BYTES[case["dtype"]] + 0.5 + 1 / 32 + 2), "flops": 0}
    if op == "transpose":
        n, out = case["rows"] * case["cols"], padded(case["rows"]) * case["cols"]
        source = BYTES.get(case["source"], 1 + 1 / 32)
        return {"bytes": n * source + out * (code[case["to"]] + 1 / 32 + 2), "flops": 0}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k * (code[case["a"]] + 1 / 32) + n * k * (0.5 + 1 / 32) + m * n * 2, "flops": 2 * m * n * k}
    n, size, train = case["rows"] * case["cols"], BYTES[case["dtype"]], case["pass"] == "train"
    kept = 1 + 1 / 32
    if op == "swiglu":
        # x and, for training, dh in; h codes and values, the kept codes, dx out
        return {"bytes": n * (2 * size + kept + 2) + (n * (2 * kept + size + 2 * size) if train else 0), "flops": 0}
    return {"bytes": n * (size + kept + 2) + case["cols"] * 4 + (n * (kept + 2 * size) + case["cols"] * 4 if train else 0),
            "flops": 0}


# ------------------------------------------------------- formats, in elementary operations

def times_pow2(v, e):
    """v 2^e for whole e, exactly (the factor is put together from its bits)."""
    if v.dtype == torch.float64:
        return v * ((e.long() + 1023) << 52).view(torch.float64)
    return v * ((e.int() + 127).clamp(1, 254) << 23).view(torch.float32)


def block_exponents(amax, fmt, rule):
    """E8M0 exponents of fp32 block maxima.  frexp: amax = m 2^p, m in [0.5, 1)."""
    m, p = torch.frexp(amax)
    emax = {"e2m1": 2, "e4m3": 8, "e5m2": 15}[fmt]
    e = p - 1 - emax
    if rule == "ceil":
        e = e + (m > FORMATS[fmt][2] / 2.0 ** (emax + 1)).to(e.dtype)
    return torch.where(amax == 0, torch.full_like(e, -127), e.clamp(-127, 127))


def round_to(v, fmt):
    """fp32 values rounded (to nearest, ties to even) to the values of fmt, saturated."""
    mantissa, emin, top = FORMATS[fmt]
    _, p = torch.frexp(v)
    quantum = (p - 1).clamp(min=emin) - mantissa
    return times_pow2(torch.round(times_pow2(v, -quantum)), quantum).clamp(-top, top)


def blocks_of(x, fmt, rule):
    """fp32 [rows][cols] -> (elements in units of their scales, exponents [rows][cols / 32])."""
    rows, cols = x.shape
    b = x.view(rows, cols // 32, 32)
    e = block_exponents(b.abs().amax(-1), fmt, rule)
    return round_to(times_pow2(b, -e.unsqueeze(-1)), fmt).view(rows, cols), e


def scaled(v, e):
    rows, cols = v.shape
    return times_pow2(v.view(rows, cols // 32, 32), e.unsqueeze(-1)).view(rows, cols)


def rounded(x, fmt, rule):
    """The values that x's codes stand for, in fp32."""
    return scaled(*blocks_of(x, fmt, rule))


def code_values(fmt, device):
    """fp32 value of each code."""
    if fmt == "e2m1":
        half = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=device)
        return torch.cat([half, -half])
    mantissa, emin, top = FORMATS[fmt]
    c = torch.arange(256, device=device)
    field, frac = (c & 127) >> mantissa, (c & (1 << mantissa) - 1).float()
    size = torch.where(field == 0, frac * 2.0 ** (emin - mantissa),
                       times_pow2(frac + (1 << mantissa), field + emin - 1 - mantissa))
    size = torch.where(size > top, torch.zeros_like(size), size)  # the specials: no input holds one
    return torch.where(c >= 128, -size, size)


def as_codes(v, e, fmt):
    """Elements in units of their scales -> code bytes (E2M1: two to a byte, the even column low), scale bytes."""
    if fmt == "e2m1":
        mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
        c = (torch.bucketize(v.abs(), mid) | (torch.signbit(v).int() << 3)).to(torch.uint8)
        q = c[:, 0::2] | (c[:, 1::2] << 4)
    else:
        q = v.to(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).view(torch.uint8)
    return q.contiguous(), (e + 127).to(torch.uint8)


def decoded(q, s, fmt, dtype=torch.float32):
    """Codes and scale bytes -> the values they stand for."""
    table = code_values(fmt, q.device).to(dtype)
    if fmt == "e2m1":
        i = torch.stack((q & 15, q >> 4), -1).view(q.shape[0], -1).int()
    else:
        i = q.int()
    return scaled(table[i], s.int() - 127)


# ----------------------------------------------------------------------------- inputs

def activations(gen, rows, cols, dtype):
    """N(0, 1) with per-channel factors in [0.1, 30], as hidden states have them."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    factor = torch.empty(cols, device="cuda").uniform_(-2.3, 3.4, generator=gen).exp_()
    return x.mul_(factor).to(dtype)


def operand(gen, rows, cols, fmt, spread):
    return as_codes(*blocks_of(torch.randn(rows, cols, generator=gen, device="cuda") * spread, fmt, "ceil"), fmt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, state = case["op"], {"case": case}
    if op == "gemm":
        state["a"], state["sa"] = operand(gen, case["m"], case["k"], case["a"], 1e-3 if case["a"] == "e5m2" else 1.0)
        state["b"], state["sb"] = operand(gen, case["n"], case["k"], "e2m1", 0.02)
        return state
    rows, cols = case["rows"], case["cols"]
    if op == "transpose" and case["source"] in FORMATS:
        x = activations(gen, rows, cols, torch.float32)
        state["q"], state["s"] = as_codes(*blocks_of(x, case["source"], "ceil"), case["source"])
        return state
    dtype = DTYPES[case["source"] if op == "transpose" else case["dtype"]]
    if op == "swiglu":
        state["x"] = torch.randn(rows, 2 * cols, generator=gen, device="cuda").mul_(2.0).to(dtype)
        state["dh"] = torch.randn(rows, cols, generator=gen, device="cuda").mul_(1e-3).to(dtype)
    elif op == "rmsnorm":
        state["x"] = activations(gen, rows, cols, dtype)
        state["w"] = torch.randn(cols, generator=gen, device="cuda").mul_(0.1).add_(1.0)
        state["dy"] = torch.randn(rows, cols, generator=gen, device="cuda").mul_(1e-3).to(dtype)
    elif op == "quantize" and rows == 1:
        state["x"] = activations(gen, rows, cols, dtype)
    else:
        state["x"] = torch.randn(rows, cols, generator=gen, device="cuda").mul_(0.02).to(dtype)
    return state


# ------------------------------------------------------------------------- plain forms

def plain_quantize(case, x):
    return rounded(x.float(), "e2m1", case["rule"]).to(torch.bfloat16)


def plain_transpose(case, state):
    x = decoded(state["q"], state["s"], case["source"]) if "q" in state else state["x"].float()
    t = torch.zeros(case["cols"], padded(case["rows"]), device=x.device)
    t[:, : case["rows"]] = x.t()
    return rounded(t, case["to"], case["rule"]).to(torch.bfloat16)


def plain_gemm(case, state):
    a = decoded(state["a"], state["sa"], case["a"])
    b = decoded(state["b"], state["sb"], "e2m1")
    return torch.matmul(a, b.t()).to(torch.bfloat16)


def plain_swiglu(case, state):
    x = state["x"].float()
    g, u = x.chunk(2, dim=1)
    h = rounded(g / (1 + torch.exp(-g)) * u, "e4m3", "ceil").to(torch.bfloat16)
    if case["pass"] == "serve":
        return {"h": h}
    g, u = rounded(x, "e4m3", "ceil").chunk(2, dim=1)
    s, dh = 1 / (1 + torch.exp(-g)), state["dh"].float()
    dx = torch.cat((dh * u * s * (1 + g * (1 - s)), dh * g * s), dim=1)
    return {"h": h, "dx": dx.to(state["x"].dtype)}


def plain_rmsnorm(case, state):
    x, w = state["x"].float(), state["w"]
    r = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    y = rounded(x * r * w, "e4m3", "ceil").to(torch.bfloat16)
    if case["pass"] == "serve":
        return {"y": y}
    xh, dy = rounded(x, "e4m3", "ceil") * r, state["dy"].float()
    c = dy * w
    dx = r * (c - xh * (c * xh).mean(1, keepdim=True))
    return {"y": y, "r": r[:, 0], "dx": dx.to(state["x"].dtype), "dw": (dy * xh).sum(0)}


# ------------------------------------------------------------------- the library's calls

def own_quantize(mx, case, x):
    q, s = mx.quantize_mxfp4(x, mx.RULE_CEIL if case["rule"] == "ceil" else mx.RULE_FLOOR)
    return mx.dequantize_mx(q, s, mx.E2M1, torch.bfloat16)


def own_transpose(mx, case, state):
    fmt = {"e2m1": mx.E2M1, "e4m3": mx.E4M3, "e5m2": mx.E5M2}
    to, rule = fmt[case["to"]], mx.RULE_CEIL if case["rule"] == "ceil" else mx.RULE_FLOOR
    if "q" in state:
        q, s = mx.requantize_mx_t(state["q"], state["s"], fmt[case["source"]], to, rule)
    else:
        q, s = mx.quantize_mx_t(state["x"], to, rule)
    return mx.dequantize_mx(q, s, to, torch.bfloat16)


def own_gemm(mx, case, state):
    fmt = {"e2m1": mx.E2M1, "e4m3": mx.E4M3, "e5m2": mx.E5M2}[case["a"]]
    return mx.mxfp4_scaled_gemm(state["a"], state["sa"], fmt, state["b"], state["sb"], out_dtype=torch.bfloat16)


def own_swiglu(mx, case, state):
    train = case["pass"] == "train"
    h, hs, kept = mx.swiglu_mx(state["x"], keep=train)
    out = {"h": mx.dequantize_mx(h, hs, mx.E4M3, torch.bfloat16)}
    if train:
        out["dx"] = mx.swiglu_mx_backward(kept, state["dh"])
    return out


def own_rmsnorm(mx, case, state):
    train = case["pass"] == "train"
    y, ys, kept = mx.rmsnorm_mx(state["x"], state["w"], EPS, keep=train)
    out = {"y": mx.dequantize_mx(y, ys, mx.E4M3, torch.bfloat16)}
    if train:
        out["r"] = kept.rstd
        out["dx"], out["dw"] = mx.rmsnorm_mx_backward(kept, state["w"], state["dy"])
    return out


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import mx_block_scaled_x128_amd as mx

        if op == "quantize":
            return own_quantize(mx, case, state["x"])
        return {"transpose": own_transpose, "gemm": own_gemm, "swiglu": own_swiglu, "rmsnorm": own_rmsnorm}[op](
            mx, case, state)
    if op == "quantize":
        return plain_quantize(case, state["x"])
    return {"transpose": plain_transpose, "gemm": plain_gemm, "swiglu": plain_swiglu, "rmsnorm": plain_rmsnorm}[op](
        case, state)


# ------------------------------------------------------------- the definition, in 64 bits

def nearest(x, fmt, rule):
    """The values of x's codes (float64), by the definition: the exponent from the real
    logarithm's bounds by comparison, the element by search among the format's values."""
    rows, cols = x.shape
    values = sorted({abs(float(v)) for v in code_values(fmt, "cpu")})
    grid = torch.tensor(values, dtype=torch.float64, device=x.device)
    emax = {"e2m1": 2, "e4m3": 8, "e5m2": 15}[fmt]
    b = x.view(rows, cols // 32, 32)
    amax = b.abs().amax(-1)
    power = torch.arange(-127, 128, device=x.device)
    bound = times_pow2(grid[-1], power) if rule == "ceil" else times_pow2(grid.new_ones(()), power[1:] + emax)
    # ceil: the first exponent whose largest value is not below amax; floor: the first whose next binade is above it
    e = torch.searchsorted(bound, amax, right=rule == "floor").clamp(max=254) - 127
    v = times_pow2(b, -e.unsqueeze(-1))
    size = v.abs().clamp(max=float(grid[-1])).contiguous()
    up = torch.searchsorted(grid, size).clamp(max=len(values) - 1)
    low = (up - 1).clamp(min=0)
    below, above = size - grid[low], grid[up] - size
    pick = torch.where((below < above) | ((below == above) & (low % 2 == 0)), low, up)
    return times_pow2(torch.copysign(grid[pick], v), e.unsqueeze(-1)).view(rows, cols)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return nearest(state["x"].double(), "e2m1", case["rule"])
    if op == "transpose":
        x = decoded(state["q"], state["s"], case["source"], torch.float64) if "q" in state else state["x"].double()
        t = torch.nn.functional.pad(x, (0, 0, 0, padded(case["rows"]) - case["rows"]))
        return nearest(t.t().contiguous(), case["to"], case["rule"])
    if op == "gemm":
        a = decoded(state["a"], state["sa"], case["a"], torch.float64)
        b = decoded(state["b"], state["sb"], "e2m1", torch.float64)
        return a @ b.t()
    x = state["x"].double()
    if op == "swiglu":
        half = case["cols"]
        h = nearest(x[:, :half] * torch.sigmoid(x[:, :half]) * x[:, half:], "e4m3", "ceil")
        if case["pass"] == "serve":
            return {"h": h}
        kept = nearest(x, "e4m3", "ceil")
        del x
        g, u, dh = kept[:, :half], kept[:, half:], state["dh"].double()
        s = torch.sigmoid(g)
        dx = torch.empty_like(kept)
        dx[:, :half] = dh * u * (s + g * s * torch.sigmoid(-g))
        dx[:, half:] = dh * (g * s)
        return {"h": h, "dx": dx}
    w = state["w"].double()
    r = 1 / torch.sqrt(torch.linalg.vector_norm(x, dim=1) ** 2 / case["cols"] + EPS)
    y = nearest(x * r[:, None] * w, "e4m3", "ceil")
    if case["pass"] == "serve":
        return {"y": y}
    xh, c = nearest(x, "e4m3", "ceil") * r[:, None], state["dy"].double() * w
    dot = (c * xh).sum(1) / case["cols"]
    return {"y": y, "r": r, "dx": (c - xh * dot[:, None]) * r[:, None],
            "dw": (state["dy"].double() * xh).sum(0)}
