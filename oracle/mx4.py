"""Microscaled 4-bit floating point in fp64: e2m1 elements, one power-of-two
scale per 32 columns (OCP Microscaling Formats v1.0, MXFP4), after the codec's
channel scale and block Hadamard rotation. Test infrastructure only.

An element code has a sign (bit 3), an exponent (bits 2-1, bias 1) and a
mantissa (bit 0): magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 for codes 0..7. A group
of 32 columns has the exponent e = clamp(floor(log2 max|y|) - 2, -127, 127)
(2 is the exponent of the largest element), stored as e + 127; every element is
the one nearest y 2^-e, ties to the even code, magnitudes above 6 to 6.
"""
from __future__ import annotations

import numpy as np

from . import codec

GROUP = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def prepare_rows(W, s, divide: bool, block: int, seed: int) -> np.ndarray:
    """y = H_b (d * (w s or w / s)) / sqrt(b), or the scaled rows for block 0 (fp64 [M, K])."""
    Y = np.asarray(W, dtype=np.float64)
    if s is not None:
        s64 = np.asarray(s, dtype=np.float64)
        Y = Y / s64 if divide else Y * s64
    return codec.rotate_fwd(Y, codec.sign_mask(seed, Y.shape[1]), block) if block else Y


def quantize_rows(Y):
    """(codes uint8 [M, K], scale bytes uint8 [M, K/32], margin [M, K]) of fp64
    rows; margin is the distance of y 2^-e to the nearest rounding border."""
    M, K = Y.shape
    G = Y.reshape(M, K // GROUP, GROUP)
    finite = np.isfinite(G).all(axis=2)
    Z = np.where(finite[:, :, None], G, 0.0)
    top = np.abs(Z).max(axis=2)
    e = np.full(top.shape, -127, dtype=np.int64)
    nz = top > 0
    e[nz] = np.clip(np.frexp(top[nz])[1] - 1 - 2, -127, 127)     # frexp: top = f 2^n, f in [1/2, 1)
    a = np.ldexp(np.abs(Z), -e[:, :, None])
    borders = (MAGNITUDES[1:] + MAGNITUDES[:-1]) / 2
    code = np.zeros(a.shape, dtype=np.int64)
    for k, b in enumerate(borders):        # code k -> k + 1 above the border, at the border if k + 1 is even
        code += (a > b) | ((a == b) & ((k + 1) % 2 == 0))
    margin = np.abs(a[..., None] - borders).min(axis=-1)
    code |= np.where(np.signbit(Z), 8, 0)
    byte = np.where(finite, e + 127, 255).astype(np.uint8)
    code = np.where(finite[:, :, None], code, 0)
    return code.reshape(M, K).astype(np.uint8), byte, margin.reshape(M, K)


def pack_codes(code) -> np.ndarray:
    """[M, K] codes -> uint8 [M, K/2], the even column in the low half."""
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def unpack_codes(packed) -> np.ndarray:
    M, H = packed.shape
    out = np.empty((M, 2 * H), dtype=np.uint8)
    out[:, 0::2] = packed & 15
    out[:, 1::2] = packed >> 4
    return out


def values(code, byte) -> np.ndarray:
    """The numbers that codes [M, K] and scale bytes [M, K/32] stand for (fp64; NaN for byte 255)."""
    v = MAGNITUDES[code & 7] * np.where(code & 8, -1.0, 1.0)
    scale = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    return v * np.repeat(scale, GROUP, axis=1)


def decode(code, byte, s, divide: bool, block: int, seed: int) -> np.ndarray:
    """The matrix in its original basis (fp64 [M, K])."""
    X = values(code, byte)
    if block:
        X = codec.rotate_inv(X, codec.sign_mask(seed, X.shape[1]), block)
    if s is not None:
        s64 = np.asarray(s, dtype=np.float64)
        X = X * s64 if divide else X / s64
    return X


def tile_scales(byte) -> np.ndarray:
    """Scale bytes [M, G] in tiles of 128 rows x 4 groups (512 bytes each),
    row tiles outermost; padding 0."""
    M, G = byte.shape
    mt, kt = -(-M // 128), -(-G // 4)
    full = np.zeros((mt * 128, kt * 4), dtype=np.uint8)
    full[:M, :G] = byte
    # (tile row, r / 32, r % 32, tile column, g) -> (tile row, tile column, r % 32, r / 32, g)
    return full.reshape(mt, 4, 32, kt, 4).transpose(0, 3, 2, 1, 4).reshape(-1)
