"""GPU parity of the MXFP4 quantizer and its inverse with the FP64 oracle:
codes, scale bytes and values bit-exact (they are decisions and exact products,
so there is no tolerance)."""

import numpy as np
import pytest
import torch

import lora_gemm_b200 as lg
from oracle import mxfp4 as o4

pytestmark = pytest.mark.gpu
DEV = "cuda"


def scale_offsets(rows, K):
    """Byte offsets of the scales of rows 0..rows-1 in the blocked layout."""
    kb, r = np.arange(K // 32)[None, :], np.arange(rows)[:, None]
    return ((r // 128) * (K // 128) + kb // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + kb % 4


def _check(x):
    rows, K = x.shape
    codes, scales = lg.mxfp4_quantize(x.to(DEV))
    c, s = o4.mx_quantize(x.float().numpy().astype(np.float64))
    assert np.array_equal(codes.cpu().numpy(), o4.pack(c))
    got = scales.cpu().numpy()
    assert np.array_equal(got[scale_offsets(rows, K)], s)
    padded = -(-rows // 128) * 128
    assert (got[scale_offsets(padded, K)[rows:]] == 0).all()
    values = lg.mxfp4_dequantize(codes, scales).float().cpu().numpy().astype(np.float64)
    want = o4.mx_dequantize(c, s)
    assert np.array_equal(values, want, equal_nan=True)


@pytest.mark.parametrize("rows,K", [(1, 128), (127, 256), (300, 1024), (129, 7168), (1000, 384)])
def test_bit_exact(rows, K):
    g = torch.Generator().manual_seed(rows * 13 + K)
    x = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g).float())
    _check(x.to(torch.bfloat16))


def test_special_blocks():
    """Every midpoint and both its bf16 neighbours, zeros, the type's ends, NaN and infinities."""
    x = torch.zeros(14, 128)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    x[0, :8], x[0, 8:16], x[0, 16] = mids, -mids, 6.0
    x[1, :8], x[1, 8:16], x[1, 16] = mids * (1 + 2.0 ** -7), mids * (1 - 2.0 ** -8), 4.0
    x[2, :32] = -0.0
    x[3, 32:64] = 2.0 ** -130                   # exponent clamped at -127
    x[4, 64:96] = -(2.0 ** 127)
    x[5, 0] = float("nan")
    x[6, 127] = float("inf")
    x[7, 31], x[7, 32] = -float("inf"), 1.0     # the next block stays
    x[8] = torch.finfo(torch.bfloat16).max
    x[9] = torch.finfo(torch.bfloat16).min
    x[10] = torch.finfo(torch.bfloat16).tiny
    x[11] = 2.0 ** -133                         # the smallest bf16 subnormal
    x[12, 0], x[12, 1:32] = 2.0 ** 100, 2.0 ** -100
    x[13, 5] = 1.0
    _check(x.to(torch.bfloat16))


def test_every_bf16_value():
    """All 65,536 bf16 bit patterns, each beside a block maximum that keeps it on the grid."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.zeros(65536 // 64, 64 * 2, dtype=torch.bfloat16)
    x[:, 0::2] = bits.view(-1, 64)
    _check(x)


def test_empty_and_reused_buffers():
    codes, scales = lg.mxfp4_quantize(torch.empty(0, 256, dtype=torch.bfloat16, device=DEV))
    assert codes.shape == (0, 128) and lg.mxfp4_dequantize(codes, scales).shape == (0, 256)
    x = torch.randn(70, 256, device=DEV).to(torch.bfloat16)
    codes = torch.full((70, 128), 9, dtype=torch.uint8, device=DEV)
    scales = torch.full((128 * 8 + 64,), 7, dtype=torch.uint8, device=DEV)
    lg.mxfp4_quantize(x, codes, scales)
    ref = lg.mxfp4_quantize(x)
    assert torch.equal(codes, ref[0]) and torch.equal(scales[:1024], ref[1])
    assert (scales[1024:] == 7).all()  # past the blocked layout nothing is written
