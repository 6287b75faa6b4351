"""The 4-bit KV format for the oracle: E2M1 codes with one E4M3 scale for 16
values, packed into pool rows.

Test infrastructure only (see ``oracle/__init__``).

Definition: E2M1 is 1 sign bit, 2 exponent bits with bias 1 and 1 mantissa bit
(exponent 0 is subnormal), i.e. 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives.  A stored element is scale * sf * code value, with sf the E4M3
scale of its block of 16 consecutive elements and ``scale`` one number per
pool.  A pool row keeps heads in blocks of four: the block's codes (element 2i
of a head in the low half of its byte i), then the block's scales; rows are
padded to a multiple of 16 bytes.
"""

import numpy as np

from .fp8 import e4m3_to_float, float_to_e4m3

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_to_float(codes):
    c = np.asarray(codes, dtype=np.int64)
    return np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]


def float_to_e2m1(x):
    """The nearest E2M1 code, a tie going to the even code, magnitudes beyond 6 to 6 (written as a search)."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 7.0)      # (an infinity is beyond 6 like any other)
    d = np.abs(a[..., None] - MAGNITUDES)
    best = d.min(-1, keepdims=True)
    near = d == best
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    return (code + 8 * np.signbit(x)).astype(np.uint8)


def row_bytes(kv_heads, d):
    n = kv_heads * (d // 2 + d // 16)
    return -(-n // 16) * 16


def quantise(x, scale):
    """(E2M1 codes [..., d], E4M3 scale codes [..., d / 16]) of x, quotients in float32 as the write path takes them."""
    x = np.asarray(x, dtype=np.float32)
    b = x.reshape(x.shape[:-1] + (-1, 16))
    nan = np.isnan(b).any(-1)
    with np.errstate(all="ignore"):
        amax = np.max(np.abs(b), -1)
        q = amax / (np.float32(6) * np.float32(scale))
        sf = float_to_e4m3(np.where(nan, np.nan, q.astype(np.float64))) & 0x7F
        f = (e4m3_to_float(sf).astype(np.float32) * np.float32(scale))[..., None]
        y = np.where(f > 0, b / f, np.copysign(np.float32(0), b))
    codes = float_to_e2m1(np.where(np.isnan(y), 0.0, y))
    return codes.reshape(x.shape), sf.astype(np.uint8)


def pack(codes, sf):
    """Pool rows [n, row_bytes] of codes [n, heads, d] and scales [n, heads, d / 16]."""
    n, heads, d = codes.shape
    rows = np.zeros((n, row_bytes(heads, d)), dtype=np.uint8)
    at = 0
    for h0 in range(0, heads, 4):
        for h in range(h0, min(heads, h0 + 4)):
            rows[:, at:at + d // 2] = codes[:, h, 0::2] | (codes[:, h, 1::2] << 4)
            at += d // 2
        for h in range(h0, min(heads, h0 + 4)):
            rows[:, at:at + d // 16] = sf[:, h]
            at += d // 16
    return rows


def unpack(rows, heads, d):
    """(codes [n, heads, d], scales [n, heads, d / 16]) of pool rows."""
    n = rows.shape[0]
    codes = np.zeros((n, heads, d), dtype=np.uint8)
    sf = np.zeros((n, heads, d // 16), dtype=np.uint8)
    at = 0
    for h0 in range(0, heads, 4):
        for h in range(h0, min(heads, h0 + 4)):
            codes[:, h, 0::2] = rows[:, at:at + d // 2] & 15
            codes[:, h, 1::2] = rows[:, at:at + d // 2] >> 4
            at += d // 2
        for h in range(h0, min(heads, h0 + 4)):
            sf[:, h] = rows[:, at:at + d // 16]
            at += d // 16
    return codes, sf


def values(rows, heads, d, scale):
    """Float64 values [n, heads, d] of pool rows."""
    codes, sf = unpack(rows, heads, d)
    return e2m1_to_float(codes) * np.repeat(e4m3_to_float(sf), 16, -1) * float(scale)


class Fp4View:
    """Float64 rows of a 4-bit pool (uint8 array [S, row bytes])."""

    def __init__(self, rows, heads, d, scale):
        self.rows, self.heads, self.d, self.scale = rows, heads, d, scale

    def __getitem__(self, slots):
        return values(self.rows[np.asarray(slots, dtype=np.int64)], self.heads, self.d, self.scale)
