"""MXFP4 in float64: E2M1 codes with one UE8M0 scale per 32 K elements (OCP
Microscaling Formats specification 1.0), the library's quantization rule and
its scale-word layout.  Test infrastructure only."""

from __future__ import annotations

import numpy as np

# code -> value: sign bit, two exponent bits (bias 1), one mantissa bit
VALUES = np.array([(1 - 2 * (c >> 3)) * (((c & 1) / 2) if (c >> 1) & 3 == 0 else
                                         (1 + (c & 1) / 2) * 2.0 ** (((c >> 1) & 3) - 1))
                   for c in range(16)])


def encode_rne(v: np.ndarray) -> np.ndarray:
    """Codes of the nearest values (ties to the even code), saturating at 6; the
    sign of a value that rounds to zero is kept."""
    v = np.asarray(v, np.float64)
    mag = np.abs(v)[..., None]
    dist = np.abs(mag - VALUES[:8])
    best = dist.min(-1, keepdims=True)
    near = dist == best
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(near.sum(-1, keepdims=True) > 1, even, near)
    return (pick.argmax(-1) | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)


def scale_exponent(amax: np.ndarray) -> np.ndarray:
    """The smallest e >= -127 with 6 * 2^e >= amax."""
    amax = np.asarray(amax, np.float64)
    e = np.full(amax.shape, -127, np.int64)
    frac, ex = np.frexp(amax)  # amax = frac 2^ex, 6 = 0.75 * 2^3
    cand = ex - 3 + (frac > 0.75)
    return np.where(amax > 0, np.maximum(cand, -127), e)


def quantize(x: np.ndarray):
    """x float32 [.., R, K] -> (codes uint8 [.., R, K], scale bytes uint8 [.., R,
    K/32]); a group with an infinity or a NaN: byte 255, codes 0."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    e = scale_exponent(np.abs(g).max(-1))
    codes = encode_rne(np.ldexp(g, -e[..., None]))
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    byte = np.where(bad, 255, e + 127).astype(np.uint8)
    return codes.reshape(x.shape), byte


def pack(codes: np.ndarray) -> np.ndarray:
    """Two codes per byte, the even element in the low nibble."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(q: np.ndarray) -> np.ndarray:
    return np.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)


def values(codes: np.ndarray, byte: np.ndarray) -> np.ndarray:
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    return VALUES[codes] * np.repeat(s, 32, -1)


def scale_words(byte: np.ndarray) -> np.ndarray:
    """Scale bytes [R, K/32] -> int32 words [ceil(R/128), ceil(K/128), 32, 4], element
    by element from the definition; zeros past R and K."""
    r, kg = byte.shape
    rb, kw = -(-r // 128), -(-kg // 4)
    out = np.zeros((rb, kw, 32, 4), np.uint32)
    for i in range(r):
        for g in range(kg):
            out[i // 128, g // 4, i % 32, (i % 128) // 32] |= np.uint32(byte[i, g]) << np.uint32(
                8 * (g % 4))
    return out.view(np.int32)


def gemm_f64(a: np.ndarray, b: np.ndarray) -> np.ndarray:
    """A B^T of two operands' values."""
    return a @ b.T
