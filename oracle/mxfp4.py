"""fp64 oracle of the microscaled 4-bit format (MXFP4), in plain numpy.

TEST INFRASTRUCTURE ONLY, like ``oracle.oracle``: it shares no code with the
product.  Values travel as float64 (fp32 where a rounding is part of the
definition), bf16 as uint16 bit patterns, codes as numbers 0..15 and scales as
bytes e + 127 (255: NaN).
"""
from __future__ import annotations

import numpy as np

from . import oracle as O

MXFP4_G32 = 16
MXFP4A4_G32 = 17
CODE_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
CODE_VALUES = np.concatenate([CODE_VALUES, -CODE_VALUES])


def bf16_values(bits: np.ndarray) -> np.ndarray:
    return (np.ascontiguousarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def rotated(v: np.ndarray) -> np.ndarray:
    """The fp32 rotation of each 128 columns, by the oracle's own transform."""
    b = np.ascontiguousarray(v, np.float32).reshape(-1, 128)
    return np.array([O.fwht128_spec_f32(r) for r in b], np.float32).reshape(v.shape)


def quantise(v: np.ndarray, rotate: bool = False):
    """(code numbers [R, K] uint8, scale bytes [R, K / 32] uint8) of fp32 rows."""
    v = np.ascontiguousarray(v, np.float32)
    if rotate:
        v = rotated(v)
    g = v.reshape(v.shape[0], v.shape[1] // 32, 32).astype(np.float64)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    amax = np.abs(g).max(-1)
    _, ex = np.frexp(amax)  # amax = m 2^ex with m in [0.5, 1): floor(log2 amax) = ex - 1
    e = np.where(amax > 0, np.maximum(ex - 3, -127), -127)
    a = np.ldexp(np.abs(g), -e[..., None])
    d = np.abs(a[..., None] - CODE_VALUES[:8])
    near = d.min(-1, keepdims=True)
    tie = d == near  # one code, or two neighbours: the even one
    n = np.where(tie.sum(-1) > 1, (np.argmax(tie, -1) + 1) // 2 * 2, np.argmax(tie, -1))
    n = (n + 8 * np.signbit(g)).astype(np.uint8)
    n[bad] = 0
    byte = np.where(bad, 255, e + 127).astype(np.uint8)
    return n.reshape(v.shape), byte


def values(codes: np.ndarray, bytes_: np.ndarray) -> np.ndarray:
    s = np.where(bytes_ == 255, np.nan, np.ldexp(1.0, bytes_.astype(np.int64) - 127))
    return CODE_VALUES[codes] * np.repeat(s, 32, axis=-1)


def pack(codes: np.ndarray, bytes_: np.ndarray):
    """Packed codes [R, K / 2] and the scale bytes in 128 x 128 blocks, one byte at a time."""
    R, K = codes.shape
    out = np.zeros(((R + 127) // 128, K // 128, 32, 4, 4), np.uint8)
    for r in range(R):
        for j in range(K // 32):
            out[r // 128, j // 4, r % 32, r % 128 // 32, j % 4] = bytes_[r, j]
    return codes[:, 0::2] | (codes[:, 1::2] << 4), out


def packed_sizes(N: int, K: int):
    return N * K // 2, (N + 127) // 128 * (K // 128) * 512, 0


def activations(x_bits: np.ndarray, fmt: int, rotate: bool) -> np.ndarray:
    """What the product sees of bf16 rows (fp64); a row with a value that is not finite is NaN."""
    v = bf16_values(x_bits)
    if fmt == MXFP4A4_G32:
        return values(*quantise(v, rotate))
    if rotate:
        v = bf16_values(O.bf16_encode(rotated(v).astype(np.float64)))
    return np.where(np.isfinite(v), v, np.nan).astype(np.float64)


def forward(x_bits: np.ndarray, W: np.ndarray, fmt: int, rotate: bool = False):
    """(y, bound): x~ . W^T of a weight's values in fp64, and how far fp32 sums of it may be off.

    The tensor cores add 32 or 64 exact products at a time to an fp32 running sum.  Every such step is taken
    to lose at most 2^-22 (two roundings or truncations of 2^-23) of the largest partial sum, which
    sum |x||w| bounds; there are at most K / 32 of them for each of the two parts of x, and a few when partial
    sums meet.  16-bit activations enter as two parts whose sum is within 2^-22 of their block's largest
    magnitude."""
    x = activations(x_bits, fmt, rotate)
    K = x.shape[1]
    with np.errstate(invalid="ignore"):
        size = np.abs(x) @ np.abs(W).T
        bound = (2 * K / 32 + 8) * 2.0 ** -22 * size
        if fmt == MXFP4_G32:
            top = np.abs(x).reshape(x.shape[0], K // 32, 32).max(-1)
            bound = bound + 2.0 ** -22 * top @ np.abs(W).reshape(W.shape[0], K // 32, 32).sum(-1).T
        return x @ W.T, bound
