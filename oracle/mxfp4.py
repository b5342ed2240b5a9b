"""Oracle: MXFP4 quantisation (E2M1 codes, one power of two per 32 elements).

TEST INFRASTRUCTURE (see the package docstring).

The format is OCP Microscaling's: an E2M1 code (sign, magnitudes 0, .5, 1, 1.5,
2, 3, 4, 6) times the block's scale 2^(e - 127), e one byte (255: NaN).  The
readings: the scale is 2^(n - 2) with n the exponent of the block's largest
magnitude rounded to one mantissa bit (halfway up), at least 2^-126; codes
round to nearest, ties to the even code; a block with an infinity or a NaN has
e = 255 and codes 0.  Codes are held one per element here ([R, K]) and scale
bytes one per block ([R, K/32]); pack() gives the library's layout.  All
arithmetic is fp64, exact for these values.
"""
from __future__ import annotations

import numpy as np

F64 = np.float64
BLOCK = 32
MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_decode(codes) -> np.ndarray:
    c = np.asarray(codes, np.uint8)
    return np.where(c & 8, -1.0, 1.0) * MAGS[c & 7]


def e2m1_encode(v) -> np.ndarray:
    """Nearest E2M1 code, ties to the even code, magnitudes past 6 to 6 (finite input)."""
    v = np.asarray(v, F64)
    a = np.abs(v)
    code = np.zeros(a.shape, np.uint8)
    for i in range(1, 8):
        mid = 0.5 * (MAGS[i - 1] + MAGS[i])
        code[(a > mid) | ((a == mid) & (i % 2 == 0))] = i
    return code | (np.signbit(v).astype(np.uint8) << 3)


def scale_byte(amax) -> np.ndarray:
    """Scale byte of blocks with largest magnitude amax (NaN or inf: 255)."""
    amax = np.asarray(amax, F64)
    ok = np.isfinite(amax)
    m, n = np.frexp(np.where(ok, amax, 1.0))          # amax = m 2^n, m in [1/2, 1)
    e = n - 1 + (m >= 0.875) - 2
    e = np.where(amax == 0, -126, np.maximum(e, -126))
    return np.where(ok, e + 127, 255).astype(np.uint8)


def quantize_mxfp4(v) -> tuple:
    """v [R, K] real values, K % 32 == 0: codes uint8 [R, K], scale bytes uint8 [R, K/32]."""
    v = np.asarray(v, F64)
    R, K = v.shape
    b = v.reshape(R, K // BLOCK, BLOCK)
    with np.errstate(invalid="ignore"):
        e = scale_byte(np.abs(b).max(axis=2))         # (max passes a NaN on)
    bad = (e == 255)[:, :, None]
    q = np.where(bad, 0.0, b) / np.exp2(e.astype(F64) - 127)[:, :, None]
    return np.where(bad, 0, e2m1_encode(q)).astype(np.uint8).reshape(R, K), e


def dequantize_mxfp4(codes, e) -> np.ndarray:
    """Real values [R, K] of codes [R, K] and scale bytes [R, K/32]."""
    R, K = codes.shape
    x = np.where(e == 255, np.nan, np.exp2(e.astype(F64) - 127))
    return (e2m1_decode(codes).reshape(R, K // BLOCK, BLOCK) * x[:, :, None]).reshape(R, K)


def pack(codes, e) -> tuple:
    """The library's tensors: bytes [R, K/2] (even element low) and scale bytes [K/128, R, 4]."""
    R, K = codes.shape
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    return packed, np.ascontiguousarray(e.reshape(R, K // 128, 4).transpose(1, 0, 2))


def unpack(packed, sc) -> tuple:
    """Inverse of pack: codes [R, K] and scale bytes [R, K/32]."""
    R, half = packed.shape
    codes = np.empty((R, half * 2), np.uint8)
    codes[:, 0::2], codes[:, 1::2] = packed & 15, packed >> 4
    return codes, np.ascontiguousarray(sc.transpose(1, 0, 2)).reshape(R, half // 16)
