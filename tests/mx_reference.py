"""The microscaled operators in 64 bits, from their definitions, for the tests:
numpy only, no code shared with the library."""
from __future__ import annotations

import numpy as np

from weight_quantized_decode_block_amd import inputs as gen

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# positive finite E4M3FN values in code order: 127 codes, the largest 448
E4M3 = np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])
EMAX = {"mxfp4": 2, "mxfp8": 8}
GRID = {"mxfp4": E2M1, "mxfp8": E4M3}


def scale_values(s: np.ndarray) -> np.ndarray:
    return np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))


def code_values(q: np.ndarray, fmt: str) -> np.ndarray:
    """Element values of code bytes (two per byte for mxfp4)."""
    if fmt == "mxfp4":
        c = np.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], -1).astype(np.int64)
        v = E2M1[c & 7]
        return np.where(c & 8, -v, v)
    full = np.concatenate((E4M3, [np.nan]))
    v = full[q & 127]
    return np.where(q & 128, -v, v)


def values(q: np.ndarray, s: np.ndarray, fmt: str) -> np.ndarray:
    return code_values(q, fmt) * np.repeat(scale_values(s), 32, axis=-1)


def nearest_codes(a: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the grid value nearest to a >= 0, ties to the even index, saturated."""
    i = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo, hi = a - grid[i - 1], grid[i] - a
    up = (hi < lo) | ((hi == lo) & (i % 2 == 0))
    return np.where(up, i, i - 1)


def quantize(x: np.ndarray, fmt: str):
    """(codes, scale bytes) of rows given in float64 (exact values of their type)."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    with np.errstate(invalid="ignore"):
        amax = np.max(np.abs(b), axis=-1)
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 1.0, amax)
    e = np.where(amax > 0, np.frexp(amax)[1] - 1 - EMAX[fmt], -127)
    e = np.maximum(e, -127)
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    v = np.where(bad[..., None], 0.0, b) * np.ldexp(1.0, -e)[..., None]
    c = nearest_codes(np.abs(v), GRID[fmt]) + (8 if fmt == "mxfp4" else 128) * np.signbit(v)
    c = np.where(bad[..., None], 0, c).astype(np.uint8).reshape(x.shape)
    return (c[..., 0::2] | (c[..., 1::2] << 4)) if fmt == "mxfp4" else c, s


def bf16(x) -> np.ndarray:
    """float64 -> BF16 values, round to nearest even in one step."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)
    e = np.maximum(e, -125)  # BF16 subnormals start below 2^-126
    with np.errstate(invalid="ignore", over="ignore"):
        r = np.ldexp(np.rint(np.ldexp(x, 8 - e)), e - 8)
        r = np.where(np.abs(r) >= 2.0 ** 128, np.sign(x) * np.inf, r)
    return np.where(np.isfinite(x), r, x)


def silu(x):
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def weights(seed: int, N: int, K: int, spread: int = 3):
    """MXFP4 weights: uniform codes, scales 2^-j around 2^-6."""
    r = gen.rng(950, gen.T_W, seed)
    q = r.integers(0, 256, size=(N, K // 2), dtype=np.uint8)
    s = (127 - 6 - r.integers(0, spread, size=(N, K // 32))).astype(np.uint8)
    return q, s


def exact_activations(seed: int, M: int, K: int, fmt: str):
    """Activations whose products with weights() sum exactly in fp32: integers
    of at most 4 in steps of 1/2 at most, scales 1 or 1/2."""
    r = gen.rng(951, gen.T_A, seed)
    if fmt == "bf16":
        return gen.bf16_bits(r.integers(-8, 9, size=(M, K)) / 2.0), None
    s = (127 - r.integers(0, 2, size=(M, K // 32))).astype(np.uint8)
    if fmt == "mxfp4":
        return r.integers(0, 256, size=(M, K // 2), dtype=np.uint8), s
    c = nearest_codes(r.integers(0, 9, size=(M, K)) / 2.0, E4M3).astype(np.uint8)
    return c | (r.integers(0, 2, size=(M, K), dtype=np.uint8) << 7), s


def activations(seed: int, M: int, K: int, fmt: str):
    x = gen.bf16_values(gen.activations(952, K, M, salt=seed + 1)).astype(np.float64)
    return (gen.bf16_bits(x), None) if fmt == "bf16" else quantize(x, fmt)


def act_values(a, s, fmt: str) -> np.ndarray:
    return gen.bf16_values(a).astype(np.float64) if fmt == "bf16" else values(a, s, fmt)
