"""Plain 64-bit MXFP8 and gated feed-forward block (numpy), written from the definitions: the reference
of the GPU tests.  x_hat = E4M3(x / s) s, s = 2^(code - 127) the smallest power of two (2^-127 at
least) with amax <= 448 s, per block of 32."""
import numpy as np

from mxfp4_reference import pad128

SILU, GELU = 0, 1
EPS = 2.0 ** -24        # half a step of binary32, relative


def _value(c):
    e, m = (c >> 3) & 15, c & 7
    v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return -v if c & 128 else v


# E4M3 "fn": 0x7F and 0xFF are NaN
VALUES = np.array([np.nan if c & 127 == 127 else _value(c) for c in range(256)])
GRID = VALUES[:127]


def quantize_rows(x):
    """(codes [n][kp], scales [n][kp/32]) of x [n][k] float64."""
    n, k = x.shape
    kp = pad128(k)
    v = np.zeros((n, kp))
    v[:, :k] = x
    v = v.reshape(n, kp // 32, 32)
    bad = ~np.isfinite(v).all(-1)
    a = np.abs(np.where(bad[..., None], 0, v))
    m, e = np.frexp(a.max(-1))                       # amax = m 2^e, 1/2 <= m < 1
    p = np.where(m <= 0.875, e - 9, e - 8)           # 448 = 0.875 * 2^9
    p = np.where(m == 0, -127, np.maximum(p, -127))
    u = np.ldexp(a, -p[..., None])
    low = np.clip(np.searchsorted(GRID, u, side="right") - 1, 0, 125)
    middle = (GRID[low] + GRID[low + 1]) / 2
    up = (u > middle) | ((u == middle) & (low % 2 == 1))
    code = low + up + 128 * np.signbit(v)
    code = np.where(bad[..., None], 0, code).reshape(n, kp).astype(np.uint8)
    return code, np.where(bad, 255, p + 127).astype(np.uint8)


def decode(codes, scales):
    """Values [n][kp] in float64 (NaN where a scale code is 255)."""
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return VALUES[codes] * np.repeat(s, 32, axis=-1)


def exponent(x, act):
    """y and y' of a(x) = x / (1 + e^-y)."""
    if act == SILU:
        return x, np.ones_like(x)
    r = np.sqrt(2 / np.pi)
    return 2 * r * (x + 0.044715 * x ** 3), 2 * r * (1 + 3 * 0.044715 * x ** 2)


def activation(x, act):
    """a(x), a'(x)."""
    y, dy = exponent(x, act)
    with np.errstate(over="ignore"):
        s, t = 1 / (1 + np.exp(-y)), 1 / (1 + np.exp(y))
    return x * s, s + x * s * t * dy


def activation_error(x, act):
    """Bounds on the errors of a(x) and a'(x) computed in binary32 with exponential and reciprocal good to
    2 EPS each.  y takes up to five roundings, so e^-y is off by (5 |y| + 2) EPS relative, of which S = 1 / (1 +
    e^-y) takes the part 1 - S, and an addition and a reciprocal of its own: rho = ((1 - S) (5 |y| + 2) + 3) EPS;
    a = x S by one rounding more.  a' = S + a t y' with t = 1 - S, which S's error S rho and a rounding of less
    than EPS put off: |a y'| (S rho + EPS); the product's other factors and roundings rho + 6 EPS of it (a one,
    y' three, two products); and the sum's rounding.  The reciprocal gives normal numbers only: an S below
    2^-126, the smallest of them, is 0 (so it is where e^-y overflows, from 2^128 on), which changes a by less than
    2^-126 |x| and a' by less than 2^-126 (1 + |x| |y'|)."""
    y, dy = exponent(x, act)
    a, _ = activation(x, act)
    with np.errstate(over="ignore"):
        s, t = 1 / (1 + np.exp(-y)), 1 / (1 + np.exp(y))
    rho = (t * (5 * np.abs(y) + 2) + 3) * EPS
    tiny = 2.0 ** -126 * (1 + np.abs(x))
    part = np.abs(a * t * dy)
    slope = s * rho + np.abs(a * dy) * (s * rho + EPS) + part * (rho + 6 * EPS) + (s + part) * EPS
    return np.abs(a) * (rho + EPS) + tiny, slope + tiny * (1 + np.abs(dy))
