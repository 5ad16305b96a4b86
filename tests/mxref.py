"""Plain 64-bit implementation of the MX operators, for the tests: formats from their
definition, quantization by search among the format's values, the functions and their
gradients from their formulas."""
import numpy as np

E4M3, E5M2, E2M1 = 0, 1, 2
CEIL, FLOOR = 0, 1
EMAX = {E4M3: 8, E5M2: 15, E2M1: 2}
# mantissa bits, exponent bias, codes that are no finite value
_SHAPE = {E4M3: (3, 7, {0x7F}), E5M2: (2, 15, {0x7C, 0x7D, 0x7E, 0x7F}), E2M1: (1, 1, set())}


def pow2(e):
    """2^e for whole e, exactly (numpy's exp2 is not, on every processor)."""
    return np.ldexp(1.0, np.asarray(e).astype(np.int64))


def code_values(fmt):
    """float64 value of every code (NaN for those without a finite one)."""
    man, bias, special = _SHAPE[fmt]
    half = 8 if fmt == E2M1 else 128
    out = np.empty(2 * half)
    for c in range(half):
        e, m = c >> man, c & ((1 << man) - 1)
        v = np.nan if c in special else (m * 2.0 ** (1 - bias - man) if e == 0
                                         else ((1 << man) + m) * 2.0 ** (e - bias - man))
        out[c], out[half + c] = v, -v
    return out


def fmax(fmt):
    return np.nanmax(code_values(fmt))


def half_step(fmt):
    """Largest distance of a value from its code's, relative to the value, above the subnormal range."""
    return 2.0 ** -(_SHAPE[fmt][0] + 1)


def smallest(fmt):
    return code_values(fmt)[1]


def exponent(amax, fmt, rule):
    """The exponents by their definition, searched from below (frexp only for a first guess)."""
    amax = np.asarray(amax, dtype=np.float64)
    p = np.frexp(amax)[1]  # amax = m 2^p, m in [0.5, 1)
    if rule == FLOOR:
        e = p - 1 - EMAX[fmt]
    else:
        e = p - 2 - EMAX[fmt]
        for _ in range(3):
            e = np.where(amax > fmax(fmt) * pow2(e), e + 1, e)
    return np.where(amax == 0, -127, np.clip(e, -127, 127)).astype(np.int64)


def cast(v, fmt):
    """float64 values -> codes: nearest, ties to the even code, saturating, sign of zero kept."""
    table = code_values(fmt)
    half = len(table) // 2
    grid = table[:half][np.isfinite(table[:half])]
    a = np.minimum(np.abs(v), grid[-1])
    hi = np.minimum(np.searchsorted(grid, a), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - grid[lo], grid[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (c + half * np.signbit(v)).astype(np.uint8)


def pack(c):
    return (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    return np.stack((q & 15, q >> 4), -1).reshape(q.shape[0], -1)


def quantize(x, fmt, rule):
    """float64 [rows][cols] -> codes (E2M1 packed), scale bytes [rows][cols / 32]."""
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    e = exponent(np.abs(b).max(-1), fmt, rule)
    c = cast(b * pow2(-e)[..., None], fmt)
    c = np.where(bad[..., None], 0, c).astype(np.uint8).reshape(rows, cols)
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    return (pack(c) if fmt == E2M1 else c), s


def quantize_t(x, fmt, rule, rows_out):
    t = np.zeros((x.shape[1], rows_out))
    t[:, :x.shape[0]] = x.T
    return quantize(t, fmt, rule)


def dequantize(q, s, fmt):
    c = unpack(q) if fmt == E2M1 else q
    f = np.where(s == 255, np.nan, pow2(s.astype(np.int64) - 127))
    v = code_values(fmt)[c]
    return (v.reshape(v.shape[0], -1, 32) * f[..., None]).reshape(v.shape)


def sigmoid(g):
    return np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))


def swiglu(x):
    g, u = np.split(x, 2, axis=1)
    return g * sigmoid(g) * u


def swiglu_grad(x, dh):
    g, u = np.split(x, 2, axis=1)
    s = sigmoid(g)
    return np.concatenate((dh * u * s * (1 + g * sigmoid(-g)), dh * g * s), axis=1)


def rstd(x, eps):
    return 1 / np.sqrt((x * x).mean(1) + eps)


def rmsnorm_grad(x, r, w, dy):
    """Gradients with xh = x r; r is the forward pass's."""
    xh, c = x * r[:, None], dy * w
    return (c - xh * (c * xh).mean(1, keepdims=True)) * r[:, None], (dy * xh).sum(0)


def bf16(x):
    """float32 array rounded to bf16 values (nearest even)."""
    b = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16
    return b.astype(np.uint32).view(np.float32)
