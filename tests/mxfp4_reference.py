"""Plain 64-bit MXFP4 (numpy), written from the format's definition: the reference of the GPU
tests.  x_hat = E2M1(x / s) s, s = 2^(code - 127) per block of 32."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
VALUES = np.concatenate([GRID, -GRID])
FLOOR, CEIL = 0, 1


def pad128(k):
    return -(-k // 128) * 128


def philox_words(counters, seed):
    """Philox4x32-10 (Salmon et al., SC'11) of counters [n][4] uint32 under a 64-bit key."""
    c = [counters[:, i].astype(np.uint64) for i in range(4)]
    k0, k1, m32 = seed & 0xFFFFFFFF, seed >> 32, np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p0, p1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & m32,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & m32]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1).astype(np.uint32)


def sr_bits(n, kp, copy, seed):
    """The 16 bits of element (i, j), [n][kp]: half (e mod 2) of word ((e / 2) mod 4) of counter
    (e / 8, copy, tag), e = i kp + j."""
    blocks = np.arange(n * kp // 8, dtype=np.uint64)
    ctr = np.stack([blocks & np.uint64(0xFFFFFFFF), blocks >> np.uint64(32),
                    np.full_like(blocks, copy), np.full_like(blocks, 0x4D585352)], 1)
    w = philox_words(ctr.astype(np.uint32), seed)
    return np.stack([w & 0xFFFF, w >> 16], -1).reshape(n, kp).astype(np.int64)


def quantize_rows(x, rule=FLOOR, bits=None):
    """(nibbles [n][kp], scales [n][kp/32]) of x [n][k] float64; bits: those of stochastic
    rounding."""
    n, k = x.shape
    kp = pad128(k)
    v = np.zeros((n, kp))
    v[:, :k] = x
    v = v.reshape(n, kp // 32, 32)
    bad = ~np.isfinite(v).all(-1)
    a = np.abs(np.where(bad[..., None], 0, v))
    m, e = np.frexp(a.max(-1))                       # amax = m 2^e, 1/2 <= m < 1
    # floor: log2's integer part is e - 1; ceil: amax <= 6 * 2^p = 0.75 * 2^(p + 3)
    p = e - 3 if rule == FLOOR else np.where(m <= 0.75, e - 3, e - 2)
    p = np.where(m == 0, -127, np.maximum(p, -127))
    u = np.ldexp(a, -p[..., None])
    low = np.clip(np.searchsorted(GRID, u, side="right") - 1, 0, 6)
    frac = np.minimum((u - GRID[low]) / (GRID[low + 1] - GRID[low]), 1.0)
    if bits is None:
        up = (frac > 0.5) | ((frac == 0.5) & (low % 2 == 1))
    else:
        up = np.floor(frac * 65536) + bits.reshape(v.shape) >= 65536
    code = low + up + 8 * np.signbit(v)
    code = np.where(bad[..., None], 0, code).reshape(n, kp).astype(np.uint8)
    return code, np.where(bad, 255, p + 127).astype(np.uint8)


def pack(nibbles):
    return nibbles[:, 0::2] | (nibbles[:, 1::2] << 4)


def unpack(codes):
    return np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)


def decode(nibbles, scales):
    """Values [n][kp] in float64 (NaN where a scale code is 255)."""
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return VALUES[nibbles] * np.repeat(s, 32, axis=1)


def spans(offsets, rows):
    """Row ranges of the groups after the documented clamping."""
    got, end = [], 0
    for e in np.asarray(offsets)[1:]:
        e = max(end, min(int(e), rows))
        got.append((end, e))
        end = e
    return got


def grouped_positions(offsets, rows):
    """K position of every row in a grouped columnwise copy, and whether it is in a group."""
    pos, inside, start = np.zeros(rows, np.int64), np.zeros(rows, bool), 0
    for a, b in spans(offsets, rows):
        pos[a:b] = start + np.arange(b - a)
        inside[a:b] = True
        start += pad128(b - a)
    return pos, inside, start


def quantize_grouped_cols(x, offsets, kp, rule=FLOOR, bits=None):
    """The columnwise copy of x with blocks restarting at each group: nibbles [cols][used],
    scales [cols][used / 32], used = the positions the groups fill; bits: [cols][kp]."""
    rows, cols = x.shape
    pos, inside, used = grouped_positions(offsets, rows)
    v = np.zeros((cols, used))
    v[:, pos[inside]] = x[inside].T
    return quantize_rows(v, rule, None if bits is None else bits[:, :used])
