"""Cases for the operators of a frozen MXFP4 block that is tuned and served with low-rank
adapters: layer norm on MX codes, and the adapters of many requests beside the shared product.

A case's "op" names the operator:

  norm       y = (x - mean) / sqrt(var + eps) w + b as MX codes; with "keep" the normalised x
             as codes and 1 / sqrt(var + eps) for the backward pass
  norm-grad  the gradients of x, w and b from what is kept
  adapt      c = x W^T + (alpha x down^T) up^T, W in E2M1, x as MX codes, each row with the
             adapter that its id names (none: -1)
  tune       a training step of such a layer: c, the gradient of x, the gradients of the
             adapters; x kept as E4M3 codes, the gradient of c as E5M2 codes

`run` is one pass: with `own` false in elementary torch operations, with `own` true by the
library's calls.  Codes are returned as the values they stand for.
"""
import torch

own = False

# (mantissa bits, smallest normal exponent, largest finite value) of each element format
FORMATS = {"e2m1": (1, 0, 6.0), "e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
CODE = {"e2m1": 0.5 + 1 / 32, "e4m3": 1 + 1 / 32, "e5m2": 1 + 1 / 32}  # bytes of an element with its share of a scale
EPS = 1e-5


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # a training step's norm in front of the 7B-class up projection
        {"name": "norm-train-7b", "op": "norm", "rows": 16384, "cols": 3584, "dtype": "bf16", "fmt": "e4m3", "rule": "ceil",
         "bias": True, "keep": True},
        # one token's norm from fp32 hidden states, nothing kept: latency
        {"name": "norm-token", "op": "norm", "rows": 1, "cols": 1536, "dtype": "f32", "fmt": "e4m3", "rule": "ceil",
         "bias": True, "keep": False},
        # its backward pass in the training step
        {"name": "norm-grad-7b", "op": "norm-grad", "rows": 16384, "cols": 3584, "dtype": "bf16", "fmt": "e4m3"},
        # a short ragged batch at the 1.5B-class MLP width with fp32 gradients
        {"name": "norm-grad-odd", "op": "norm-grad", "rows": 515, "cols": 8960, "dtype": "f32", "fmt": "e4m3"},
        # decoding one request with its adapter: the 7B-class up projection
        {"name": "adapt-token-7b", "op": "adapt", "m": 1, "n": 18944, "k": 3584, "a": "e4m3", "rank": 16, "adapters": 8,
         "order": "each"},
        # a decoded batch, requests of many adapters mixed, the 7B-class down projection
        {"name": "adapt-batch-7b", "op": "adapt", "m": 61, "n": 3584, "k": 18944, "a": "e4m3", "rank": 64, "adapters": 32,
         "order": "each"},
        # a small batch with both sides in 4 bits, the 1.5B-class down projection
        {"name": "adapt-batch-odd", "op": "adapt", "m": 13, "n": 1536, "k": 8960, "a": "e2m1", "rank": 8, "adapters": 5,
         "order": "each"},
        # prefill: prompts of several requests behind each other, some without an adapter
        {"name": "adapt-prefill-7b", "op": "adapt", "m": 8192, "n": 18944, "k": 3584, "a": "e4m3", "rank": 16, "adapters": 8,
         "order": "runs"},
        # tuning one adapter of the 7B-class down projection
        {"name": "tune-7b", "op": "tune", "m": 8192, "n": 3584, "k": 18944, "rank": 16, "adapters": 1, "order": "runs"},
        # tuning one adapter of higher rank, the 1.5B-class up projection
        {"name": "tune-1p5b", "op": "tune", "m": 4096, "n": 8960, "k": 1536, "rank": 64, "adapters": 1, "order": "runs"},
        # a small ragged step over the adapters of several users
        {"name": "tune-odd", "op": "tune", "m": 515, "n": 1536, "k": 8960, "rank": 8, "adapters": 3, "order": "runs"},
    ]


def draw(rng):
    def spread(low, high):
        return int(round(low * (high / low) ** rng.random()))

    def width(low, high, step):
        return max(low, spread(low, high) // step * step)

    op = rng.choice(("norm", "norm-grad", "adapt", "adapt", "tune"))
    if op in ("norm", "norm-grad"):
        case = {"op": op, "rows": spread(1, 8192), "cols": width(32, 12288, 32), "dtype": rng.choice(("f32", "bf16")),
                "fmt": rng.choice(("e4m3", "e4m3", "e5m2"))}
        if op == "norm":
            case.update(rule=rng.choice(("ceil", "floor")), bias=rng.random() < 0.7, keep=rng.random() < 0.5)
        return case
    rank = rng.choice((8, 16, 24, 32, 64, 128))
    if op == "tune":
        return {"op": op, "m": spread(1, 8192), "n": width(128, 8960, 128), "k": width(128, 6912, 128), "rank": rank,
                "adapters": rng.choice((1, 1, 2, 5)), "order": "runs"}
    m = spread(1, 8192)
    return {"op": op, "m": m, "n": spread(16, 16384), "k": width(128, 3584, 128), "a": rng.choice(("e2m1", "e4m3", "e4m3")),
            "rank": rank, "adapters": spread(1, 48), "order": "each" if m <= 256 else "runs"}


def work(case):
    op = case["op"]
    if op == "norm":
        n, size = case["rows"] * case["cols"], BYTES[case["dtype"]]
        out = CODE[case["fmt"]] + 2  # the codes, and the values they are returned as
        return {"bytes": n * (size + out * (2 if case["keep"] else 1)) + case["cols"] * 8, "flops": 0}
    if op == "norm-grad":
        n, size = case["rows"] * case["cols"], BYTES[case["dtype"]]
        return {"bytes": n * (CODE[case["fmt"]] + 2 * size) + case["cols"] * 12, "flops": 0}
    m, n, k, r = case["m"], case["n"], case["k"], case["rank"]
    used = min(m, case["adapters"]) * r * (n + k)  # elements of the adapters that are used
    base = {"bytes": n * k * CODE["e2m1"] + used * 2, "flops": 2 * m * n * k + 2 * m * r * (n + k)}
    if op == "adapt":
        return {"bytes": base["bytes"] + m * k * CODE[case["a"]] + m * n * 2, "flops": base["flops"]}
    # both products, x and the gradient in, c, dx and the adapters' gradients out
    return {"bytes": base["bytes"] * 2 - used * 2 + m * k * (CODE["e4m3"] + 2) + m * n * (CODE["e5m2"] + 2)
            + case["adapters"] * r * (n + k) * 4, "flops": 2 * base["flops"] + 2 * m * r * (n + k)}


# ------------------------------------------------------- formats, in elementary operations

def times_pow2(v, e):
    """v 2^e for whole e, exactly (the factor is put together from its bits)."""
    if v.dtype == torch.float64:
        return v * ((e.long() + 1023) << 52).view(torch.float64)
    return v * ((e.int() + 127).clamp(1, 254) << 23).view(torch.float32)


def blocks_of(x, fmt, rule):
    """fp32 [rows][cols] -> (elements in units of their scales, exponents [rows][cols / 32])."""
    rows, cols = x.shape
    mantissa, emin, top = FORMATS[fmt]
    b = x.view(rows, cols // 32, 32)
    amax = b.abs().amax(-1)
    m, p = torch.frexp(amax)  # amax = m 2^p, m in [0.5, 1)
    emax = {"e2m1": 2, "e4m3": 8, "e5m2": 15}[fmt]
    e = p - 1 - emax
    if rule == "ceil":
        e = e + (m > top / 2.0 ** (emax + 1)).to(e.dtype)
    e = torch.where(amax == 0, torch.full_like(e, -127), e.clamp(-127, 127))
    v = times_pow2(b, -e.unsqueeze(-1))
    quantum = (torch.frexp(v)[1] - 1).clamp(min=emin) - mantissa
    v = times_pow2(torch.round(times_pow2(v, -quantum)), quantum).clamp(-top, top)
    return v.view(rows, cols), e


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
    """N(0, 1) with per-channel factors in [0.1, 30] around per-channel means, as hidden states have them."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    factor = torch.empty(cols, device="cuda").uniform_(-2.3, 3.4, generator=gen).exp_()
    mean = torch.randn(cols, generator=gen, device="cuda").add_(0.5)
    return x.mul_(factor).add_(mean).to(dtype)


def operand(gen, rows, cols, fmt, spread):
    return as_codes(*blocks_of(torch.randn(rows, cols, generator=gen, device="cuda") * spread, fmt, "ceil"), fmt)


def adapter_ids(gen, case):
    """int32 [m]: "each" row of its own, one in eight without an adapter; or "runs" of rows, the prompts
    or sequences of one adapter each, behind each other (a single adapter: all rows)."""
    m, count = case["m"], case["adapters"]
    if case["order"] == "each":
        ids = torch.randint(0, count, (m,), generator=gen, device="cuda", dtype=torch.int32)
        none = torch.rand(m, generator=gen, device="cuda") < 0.125
        return torch.where(none & (m > 1), torch.full_like(ids, -1), ids)
    if count == 1:
        return torch.zeros(m, dtype=torch.int32, device="cuda")
    runs = 2 * count
    ends = torch.randint(0, m + 1, (runs,), generator=gen, device="cuda").sort().values
    run = torch.searchsorted(ends, torch.arange(m, device="cuda"), right=True)
    own_id = torch.randint(-1, count, (runs + 1,), generator=gen, device="cuda", dtype=torch.int32)
    return own_id[run]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, state = case["op"], {"case": case}
    if op in ("norm", "norm-grad"):
        rows, cols, dtype = case["rows"], case["cols"], DTYPES[case["dtype"]]
        state["w"] = torch.randn(cols, generator=gen, device="cuda").mul_(0.1).add_(1.0)
        state["b"] = torch.randn(cols, generator=gen, device="cuda").mul_(0.1)
        x = activations(gen, rows, cols, dtype)
        if op == "norm":
            state["x"] = x
            if not case["bias"]:
                state["b"] = None
            return state
        # what the forward pass kept
        x = x.double()
        x -= x.mean(1, keepdim=True)
        r = torch.rsqrt(x.square().mean(1) + EPS)
        state["q"], state["s"] = as_codes(*blocks_of((x * r[:, None]).float(), case["fmt"], "ceil"), case["fmt"])
        state["r"] = r.float()
        state["dy"] = torch.randn(rows, cols, generator=gen, device="cuda").mul_(1e-3).to(dtype)
        return state
    m, n, k, rank, count = case["m"], case["n"], case["k"], case["rank"], case["adapters"]
    state["ids"] = adapter_ids(gen, case)
    state["down"] = torch.randn(count, rank, k, generator=gen, device="cuda").mul_(k ** -0.5).bfloat16()
    state["up"] = torch.randn(count, n, rank, generator=gen, device="cuda").mul_(0.02).bfloat16()
    state["alpha"] = torch.empty(count, device="cuda").uniform_(0.5, 2.0, generator=gen)
    w = torch.randn(n, k, generator=gen, device="cuda") * 0.02
    state["w"], state["sw"] = as_codes(*blocks_of(w, "e2m1", "ceil"), "e2m1")
    fmt = case["a"] if op == "adapt" else "e4m3"
    state["x"], state["sx"] = operand(gen, m, k, fmt, 1.0)
    if op == "tune":
        state["wt"], state["swt"] = as_codes(*blocks_of(w.t().contiguous(), "e2m1", "ceil"), "e2m1")
        state["g"], state["sg"] = operand(gen, m, n, "e5m2", 1e-3)
    return state


# ------------------------------------------------------------------------- plain forms

def plain_norm(case, state):
    x = state["x"].float()
    d = x - x.mean(1, keepdim=True)
    d = d - d.mean(1, keepdim=True)  # what the first mean's rounding left
    r = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    xh = d * r
    y = xh * state["w"] if state["b"] is None else xh * state["w"] + state["b"]
    out = {"y": rounded(y, case["fmt"], case["rule"]).to(torch.bfloat16)}
    if case["keep"]:
        out["xh"], out["r"] = rounded(xh, case["fmt"], case["rule"]).to(torch.bfloat16), r[:, 0]
    return out


def plain_norm_grad(case, state):
    xh, dy = decoded(state["q"], state["s"], case["fmt"]), state["dy"].float()
    c = dy * state["w"]
    dx = state["r"][:, None] * (c - c.mean(1, keepdim=True) - xh * (c * xh).mean(1, keepdim=True))
    return {"dx": dx.to(state["dy"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def own_slots(p, ids, count):
    """[m][rank] -> [m][count rank]: each row's values in the columns of its adapter, zeros elsewhere."""
    slot = (ids[:, None] == torch.arange(count, device=ids.device, dtype=torch.int32)).float()
    return (slot[:, :, None] * p[:, None, :]).view(p.shape[0], -1)


def plain_product(x, w, down, up, alpha, ids):
    """(c, p): all adapters' products of all rows, of which each row takes its own."""
    count, rank, k = down.shape
    slot = (ids[:, None] == torch.arange(count, device=ids.device, dtype=torch.int32)).float() * alpha
    p = ((x @ down.float().view(count * rank, k).t()).view(-1, count, rank) * slot[:, :, None]).sum(1)
    c = x @ w.t() + own_slots(p, ids, count) @ up.float().transpose(1, 2).reshape(count * rank, -1)
    return c, p


def plain_adapt(case, state):
    x, w = decoded(state["x"], state["sx"], case["a"]), decoded(state["w"], state["sw"], "e2m1")
    c, _ = plain_product(x, w, state["down"], state["up"], state["alpha"], state["ids"])
    return c.to(torch.bfloat16)


def plain_tune(case, state):
    down, up, alpha, ids = state["down"], state["up"], state["alpha"], state["ids"]
    count, rank = case["adapters"], case["rank"]
    x, g = decoded(state["x"], state["sx"], "e4m3"), decoded(state["g"], state["sg"], "e5m2")
    c, p = plain_product(x, decoded(state["w"], state["sw"], "e2m1"), down, up, alpha, ids)
    dx, u = plain_product(g, decoded(state["wt"], state["swt"], "e2m1"), up.transpose(1, 2).contiguous(),
                          down.transpose(1, 2).contiguous(), alpha, ids)
    d_down = (own_slots(u, ids, count).t() @ x).view(count, rank, -1)
    d_up = (own_slots(p, ids, count).t() @ g).view(count, rank, -1).transpose(1, 2).contiguous()
    return {"c": c.to(torch.bfloat16), "dx": dx.to(torch.bfloat16), "d_down": d_down, "d_up": d_up}


# ------------------------------------------------------------------- the library's calls

def own_norm(mx, case, state):
    fmt = {"e4m3": mx.E4M3, "e5m2": mx.E5M2}[case["fmt"]]
    rule = mx.RULE_CEIL if case["rule"] == "ceil" else mx.RULE_FLOOR
    y, ys, kept = mx.layernorm_mx(state["x"], state["w"], state["b"], EPS, fmt, rule, keep=case["keep"])
    out = {"y": mx.dequantize_mx(y, ys, fmt, torch.bfloat16)}
    if case["keep"]:
        out["xh"], out["r"] = mx.dequantize_mx(kept.codes, kept.scales, fmt, torch.bfloat16), kept.rstd
    return out


def own_norm_grad(mx, case, state):
    kept = mx.LayernormKept(state["q"], state["s"], state["r"], {"e4m3": mx.E4M3, "e5m2": mx.E5M2}[case["fmt"]])
    dx, dw, db = mx.layernorm_mx_backward(kept, state["w"], state["dy"])
    return {"dx": dx, "dw": dw, "db": db}


def own_adapt(mx, case, state):
    c, _ = mx.mxfp4_adapted_gemm(state["x"], state["sx"], mx.E4M3 if case["a"] == "e4m3" else mx.E2M1, state["w"],
                                 state["sw"], state["down"], state["up"], state["ids"], state["alpha"],
                                 out_dtype=torch.bfloat16)
    return c


def own_tune(mx, case, state):
    down, up, alpha, ids = state["down"], state["up"], state["alpha"], state["ids"]
    x, g = (state["x"], state["sx"], mx.E4M3), (state["g"], state["sg"], mx.E5M2)
    c, p = mx.mxfp4_adapted_gemm(*x, state["w"], state["sw"], down, up, ids, alpha, out_dtype=torch.bfloat16)
    # the data gradient is the same product with the adapters' parts transposed and in each other's place
    dx, u = mx.mxfp4_adapted_gemm(*g, state["wt"], state["swt"], up.transpose(1, 2).contiguous(),
                                  down.transpose(1, 2).contiguous(), ids, alpha, out_dtype=torch.bfloat16)
    return {"c": c, "dx": dx, "d_down": mx.adapter_grad_mx(u, *x, ids, case["adapters"]),
            "d_up": mx.adapter_grad_mx(p, *g, ids, case["adapters"], transposed=True)}


def run(state):
    case = state["case"]
    if own:
        import mx_block_scaled_x128_amd as mx

        return {"norm": own_norm, "norm-grad": own_norm_grad, "adapt": own_adapt, "tune": own_tune}[case["op"]](
            mx, case, state)
    return {"norm": plain_norm, "norm-grad": plain_norm_grad, "adapt": plain_adapt, "tune": plain_tune}[case["op"]](
        case, state)


# ------------------------------------------------------------- the definition, in 64 bits

def nearest(x, fmt, rule):
    """The values of x's codes (float64), by the definition: the exponent by comparison with each
    one's bound, the element by search among the format's values."""
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


def exact_product(x, w, down, up, alpha, ids):
    """c and p, adapter by adapter on the rows that are its own."""
    c = torch.matmul(x, w.transpose(0, 1))
    p = x.new_zeros(x.shape[0], down.shape[1])
    for a in range(down.shape[0]):
        rows = torch.nonzero(ids == a)[:, 0]
        p[rows] = torch.matmul(x[rows], down[a].double().transpose(0, 1)) * alpha[a].double()
        c[rows] += torch.matmul(p[rows], up[a].double().transpose(0, 1))
    return c, p


def exact_grad(p, z, ids, count):
    out = z.new_zeros(count, p.shape[1], z.shape[1])
    for a in range(count):
        rows = torch.nonzero(ids == a)[:, 0]
        out[a] = torch.matmul(p[rows].transpose(0, 1), z[rows])
    return out


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = state["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        r = 1 / torch.sqrt(var + EPS)
        xh = (x - mean) * r
        y = xh * state["w"].double() + (0 if state["b"] is None else state["b"].double())
        out = {"y": nearest(y, case["fmt"], case["rule"])}
        if case["keep"]:
            out["xh"], out["r"] = nearest(xh, case["fmt"], case["rule"]), r[:, 0]
        return out
    if op == "norm-grad":
        xh = decoded(state["q"], state["s"], case["fmt"], torch.float64)
        dy, cols = state["dy"].double(), case["cols"]
        c = dy * state["w"].double()
        dot = torch.linalg.vecdot(c, xh)[:, None] / cols
        dx = (c - c.sum(1, keepdim=True) / cols - xh * dot) * state["r"].double()[:, None]
        return {"dx": dx, "dw": (dy * xh).sum(0), "db": dy.sum(0)}
    down, up, alpha, ids = state["down"], state["up"], state["alpha"], state["ids"]
    fmt = case["a"] if op == "adapt" else "e4m3"
    x = decoded(state["x"], state["sx"], fmt, torch.float64)
    c, p = exact_product(x, decoded(state["w"], state["sw"], "e2m1", torch.float64), down, up, alpha, ids)
    if op == "adapt":
        return c
    g = decoded(state["g"], state["sg"], "e5m2", torch.float64)
    dx, u = exact_product(g, decoded(state["wt"], state["swt"], "e2m1", torch.float64), up.transpose(1, 2),
                          down.transpose(1, 2), alpha, ids)
    return {"c": c, "dx": dx, "d_down": exact_grad(u, x, ids, case["adapters"]),
            "d_up": exact_grad(p, g, ids, case["adapters"]).transpose(1, 2).contiguous()}
