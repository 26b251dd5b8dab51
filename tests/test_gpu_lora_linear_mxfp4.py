"""GPU parity of lora_linear_mxfp4 with the FP64 oracle.

Without adapters the product of MXFP4 values is exact up to FP32 accumulation
and the rounding of y to bf16: |y - ref| <= 2^-8 |ref| + K 2^-24 sum|products|
(each of the K terms may cost half an FP32 step of the running sum).  With
adapters the bf16 layer's bar applies (bf16 factors, bf16 h): relative
Frobenius error 1e-2, as for the other layers."""

import numpy as np
import pytest
import torch

import lora_gemm_b200 as lg
from oracle import mxfp4 as o4
from tests.util import rel_fro

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 1e-2


def _np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _layer(M, K, N, R, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(M, K, generator=g) * torch.exp2(torch.randn(M, 1, generator=g))).to(torch.bfloat16)
    W = (torch.randn(N, K, generator=g) * K ** -0.5).to(torch.bfloat16)
    A = (torch.randn(R, K, generator=g) * K ** -0.5).to(DEV) if R else None
    B = (torch.randn(N, R, generator=g) * 0.1).to(DEV) if R else None
    return x.to(DEV), W.to(DEV), A, B


def _run(x, W, A, B, **kw):
    y = lg.lora_linear_mxfp4(x, lg.mxfp4_quantize(x), lg.mxfp4_quantize(W), A, B, **kw)
    assert lg.get_last_device_error() == lg.LG_OK
    return y


def _check_base(y, x, W):
    xq, wq = o4.quantized(_np64(x)), o4.quantized(_np64(W))
    ref, mag = xq @ wq.T, np.abs(xq) @ np.abs(wq).T
    # Plus 2^-126, FP32's smallest normal number: a product of a row scaled by
    # 2^-120 with a column scaled by 2^-60 is near 2^-180, and neither the FP32
    # accumulator nor bf16 (smallest value 2^-133) can hold it.
    bad = np.abs(_np64(y) - ref) > 2.0 ** -8 * np.abs(ref) + x.shape[1] * 2.0 ** -24 * mag + 2.0 ** -126
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5])


BASE = [(1, 128, 32), (2, 256, 96), (7, 384, 64), (8, 1024, 320), (17, 640, 256), (33, 1152, 288), (64, 512, 1024),
        (65, 7168, 96), (100, 896, 160), (128, 1024, 96), (129, 128, 256), (256, 256, 256), (257, 384, 544), (700, 896, 1024), (1, 28672, 64)]


@pytest.mark.parametrize("M,K,N", BASE)
def test_base_term_elementwise(M, K, N):
    x, W, _, _ = _layer(M, K, N, 0, seed=M + 3 * K + N)
    _check_base(_run(x, W, None, None), x, W)


@pytest.mark.parametrize("M,K,N,R", [(1, 128, 64, 64), (3, 256, 32, 576), (16, 1024, 1024, 192), (48, 384, 320, 576),
                                     (100, 1152, 512, 192), (128, 7168, 96, 64), (130, 7168, 256, 576), (300, 7168, 96, 64), (700, 3200, 160, 576), (517, 384, 320, 576), (1000, 1024, 896, 64),
                                     (2304, 1024, 1024, 576), (1, 7168, 7168, 576)])
def test_with_adapters(M, K, N, R):
    x, W, A, B = _layer(M, K, N, R, seed=M + 3 * K + N)
    ref = o4.lora_linear_mxfp4(_np64(x), _np64(W), _np64(A), _np64(B))
    y = _np64(_run(x, W, A, B))
    assert rel_fro(y, ref) <= TOL
    assert np.linalg.norm(y - ref, axis=1).max() <= 2 * TOL * np.linalg.norm(ref, axis=1).max()


@pytest.mark.parametrize("R", range(64, 577, 64))
def test_every_rank(R):
    """Each rank picks its own column tiles for h (one to nine of 64 ranks), in both forms."""
    for M in (40, 200):
        x, W, A, B = _layer(M, 384, 160, R, seed=R + M)
        ref = o4.lora_linear_mxfp4(_np64(x), _np64(W), _np64(A), _np64(B))
        assert rel_fro(_np64(_run(x, W, A, B)), ref) <= TOL


@pytest.mark.parametrize("N", [32, 64, 160, 192, 224, 288, 480, 544, 2048])
def test_widths_around_the_tiles(N):
    """Widths that end inside tiles of 64, 128, 192 and 256 columns and inside scale groups of 128."""
    for M in (20, 260, 1100):
        x, W, _, _ = _layer(M, 384, N, 0, seed=N + M)
        _check_base(_run(x, W, None, None), x, W)


def test_many_tiles():
    """Several tiles per SM pair, a ragged last block of panels, an odd number of scale groups."""
    x, W, A, B = _layer(37 * 256 + 5, 896, 1792, 576, seed=4)
    y, y0 = _run(x, W, A, B), _run(x, W, None, None)
    rows = np.r_[0:300, 9000:9477]
    idx = torch.as_tensor(rows, device=DEV)
    ref = o4.lora_linear_mxfp4(_np64(x[idx]), _np64(W), _np64(A), _np64(B))
    assert rel_fro(_np64(y[idx]), ref) <= TOL
    _check_base(y0[idx], x[idx], W)


@pytest.mark.parametrize("M", [5, 300])
def test_extreme_scales_and_nan_blocks(M):
    """Rows and columns at both ends of the scale range; a NaN block makes its row (column) NaN and no other."""
    x, W, _, _ = _layer(M, 512, 128, 0, seed=3)
    x, W = x.clone(), W.clone()
    x[0] *= 2.0 ** 60
    x[1] *= 2.0 ** -120
    W[1] *= 2.0 ** 60
    W[2] *= 2.0 ** -60
    _check_base(_run(x, W, None, None), x, W)
    x[2, 77], W[3, 500] = float("nan"), float("inf")
    y = _run(x, W, None, None)
    nan = torch.zeros(M, 128, dtype=torch.bool)
    nan[2], nan[:, 3] = True, True
    assert torch.equal(torch.isnan(y).cpu(), nan)
    assert torch.isfinite(y.cpu()[~nan]).all()


def test_rows_behind_the_last_token_stay():
    """y is a slice of a larger buffer: the rows behind it keep their contents, also where the tile passes them."""
    for M in (3, 200):
        x, W, A, B = _layer(M, 256, 64, 64, seed=M)
        buf = torch.full((M + 64, 64), 5.0, dtype=torch.bfloat16, device=DEV)
        _run(x, W, A, B, y=buf[:M])
        assert (buf[M:] == 5.0).all()
        assert torch.equal(buf[:M], _run(x, W, A, B))


def test_x_is_not_needed_without_adapters():
    x, W, _, _ = _layer(40, 256, 64, 0, seed=2)
    y = lg.lora_linear_mxfp4(None, lg.mxfp4_quantize(x), lg.mxfp4_quantize(W), None, None)
    assert torch.equal(y, _run(x, W, None, None))
    assert lg.lora_linear_mxfp4(None, lg.mxfp4_quantize(x[:0]), lg.mxfp4_quantize(W), None, None).shape == (0, 64)


def test_wait_timeout_is_reported():
    x, W, A, B = _layer(2048, 1024, 1792, 576, seed=19)
    lg.set_wait_limit_ns(1)
    try:
        lg.lora_linear_mxfp4(x, lg.mxfp4_quantize(x), lg.mxfp4_quantize(W), A, B)
        status = lg.get_last_device_error()
    finally:
        lg.set_wait_limit_ns(0)
    assert status == lg.LG_ERR_DEVICE_TIMEOUT
    ref = o4.lora_linear_mxfp4(_np64(x), _np64(W), _np64(A), _np64(B))
    assert rel_fro(_np64(_run(x, W, A, B)), ref) <= TOL


def _adapters_alone(M, K, N, R, seed):
    """(y, the FP64 term) of a layer whose W is zero, with FP32 factors."""
    x, _, A, B = _layer(M, K, N, R, seed)
    y = _run(x, torch.zeros(N, K, dtype=torch.bfloat16, device=DEV), A, B)
    return y, (_np64(x) @ _np64(A).T) @ _np64(B).T


@pytest.mark.parametrize("M", [16, 64, 128])
def test_few_tokens_do_not_shrink_the_adapters_term(M):
    """The signed error of the adapters' term, as its share of the term.  Roundings to nearest have no sign:
    the mean of y's, each below 2^-8, over M N >= 65,536 outputs has a deviation below 2^-8 / 256 = 2^-16, and
    those of the factors and h are a thousandth of them.  2^-13 is eight deviations; factors and h cut to ten
    fraction bits towards zero would take 2^-10.5."""
    y, ref = _adapters_alone(M, 512, 4096, 64, seed=M)
    bias = float(((_np64(y) - ref) * ref).sum() / (ref * ref).sum())
    assert abs(bias) <= 2.0 ** -13, bias


@pytest.mark.parametrize("M", [5, 100, 300])
def test_non_finite_factors_stay_where_they_belong(M):
    """A NaN or an infinity in a row of B_cat makes its output column non-finite (the NaN: NaN) and leaves the other
    columns' bits; a NaN in A_cat reaches every output; a factor of 2^100 keeps its term."""
    x, W, A, B = _layer(M, 256, 160, 64, seed=M)
    want = _run(x, W, A, B)
    assert torch.isfinite(want).all()
    B2 = B.clone()
    B2[7, 3], B2[9, 60], B2[159, 0] = float("nan"), float("inf"), -float("inf")
    y = _run(x, W, A, B2)
    assert torch.isnan(y[:, 7]).all() and not torch.isfinite(y[:, [9, 159]]).any()
    keep = [n for n in range(160) if n not in (7, 9, 159)]
    assert torch.equal(y[:, keep], want[:, keep])
    A2 = A.clone()
    A2[5, 200] = float("nan")
    assert torch.isnan(_run(x, W, A2, B)).all()
    B3 = torch.zeros_like(B)
    B3[1, 1] = 2.0 ** 100
    ref = _np64(lg.lora_linear_mxfp4(None, lg.mxfp4_quantize(x), lg.mxfp4_quantize(W), None, None))
    big = _np64(_run(x, W, A, B3))
    h = _np64(x) @ _np64(A)[1]
    # Two roundings of the factors' term to bf16 or nearer, y's, and A's among K products.
    tol = 3 * 2.0 ** -8 * np.abs(h) + 2.0 ** -8 * (np.abs(_np64(x)) @ np.abs(_np64(A)[1]))
    assert (np.abs(big[:, 1] - h * 2.0 ** 100) <= tol * 2.0 ** 100).all()
    assert np.array_equal(np.delete(big, 1, 1), np.delete(ref, 1, 1))
