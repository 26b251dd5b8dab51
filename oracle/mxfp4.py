"""FP64 oracle of the MXFP4 format (OCP Microscaling: E2M1 elements, one E8M0
scale per 32 values) and of the merged-LoRA linear with an MXFP4 base term."""

import numpy as np

BLOCK = 32
E2M1_MAX = 6.0


def e2m1_decode(codes):
    """Values of E2M1 codes 0..15: sign, two exponent bits (bias 1), one mantissa bit."""
    c = np.asarray(codes).astype(np.int64)
    sign = np.where(c & 8, -1.0, 1.0)
    ex, m = (c >> 1) & 3, c & 1
    mag = np.where(ex > 0, (1.0 + 0.5 * m) * 2.0 ** (ex - 1.0), 0.5 * m)
    return sign * mag


def e2m1_encode(v):
    """Codes of FP64 values, round to nearest, ties to the even code, saturated at 6."""
    v = np.asarray(v, dtype=np.float64)
    grid = e2m1_decode(np.arange(8))
    a = np.minimum(np.abs(v), E2M1_MAX)
    hi = np.clip(np.searchsorted(grid, a), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - grid[lo], grid[hi] - a
    up = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
    code = np.where(up, hi, lo)
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def mx_quantize(x):
    """Codes [rows, K] (one per value, unpacked) and E8M0 bytes [rows, K / 32]
    of FP64 rows; a block with a NaN or an infinity gets byte 255 and codes 0."""
    x = np.asarray(x, dtype=np.float64)
    rows, K = x.shape
    v = x.reshape(rows, K // BLOCK, BLOCK)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    amax = np.abs(v).max(-1)
    _, ex = np.frexp(amax)
    e = np.where(amax > 0, np.clip(ex - 1 - 2, -127, 127), -127)
    codes = e2m1_encode(np.ldexp(v, -e[..., None]))
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8)
    return codes.reshape(rows, K), np.where(bad, 255, e + 127).astype(np.uint8)


def mx_dequantize(codes, scale_bytes):
    """FP64 values of unpacked codes [rows, K] and E8M0 bytes [rows, K / 32]."""
    codes = np.asarray(codes)
    s = np.asarray(scale_bytes).astype(np.int64)
    rows, K = codes.shape
    v = np.ldexp(e2m1_decode(codes).reshape(rows, K // BLOCK, BLOCK), (s - 127)[..., None])
    return np.where((s == 255)[..., None], np.nan, v).reshape(rows, K)


def pack(codes):
    """Two codes per byte, the even one low."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def quantized(x):
    """The values an MXFP4 copy of x stands for."""
    return mx_dequantize(*mx_quantize(x))


def lora_linear_mxfp4(x, W, A_cat, B_cat):
    """deq(Q(x)) deq(Q(W))^T + (x A_cat^T) B_cat^T in FP64."""
    y = quantized(x) @ quantized(W).T
    if A_cat is not None:
        y = y + (np.asarray(x, np.float64) @ np.asarray(A_cat, np.float64).T) @ np.asarray(B_cat, np.float64).T
    return y
