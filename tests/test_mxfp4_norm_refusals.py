"""Argument checks of the MXFP4 and block-norm entry points, made on the host
before anything is launched (no GPU: every call here is refused or empty)."""

import ctypes

import pytest

import lora_gemm_b200 as lg

L = lg.lib
INVALID, SHAPE, MISALIGNED, WORKSPACE = (lg.LG_ERR_INVALID_ARG, lg.LG_ERR_UNSUPPORTED_SHAPE, lg.LG_ERR_MISALIGNED,
                                         lg.LG_ERR_WORKSPACE)
BASE = 0x7F0000000000


def at(i, off=0):
    """Fake device addresses 64 GiB apart; never read."""
    return ctypes.c_void_p(BASE + i * (1 << 36) + off)


@pytest.mark.parametrize("fn", ["lg_mxfp4_quantize", "lg_mxfp4_dequantize"])
def test_quantizer_refusals(fn):
    def call(a=at(0), b=at(1), c=at(2), rows=10, K=256):
        return (L.lg_mxfp4_quantize(a, rows, K, b, c, None) if fn == "lg_mxfp4_quantize" else
                L.lg_mxfp4_dequantize(a, b, rows, K, c, None))

    assert call(rows=-1) == INVALID and call(K=-128) == INVALID
    for K in (0, 64, 96, 200, (1 << 20) + 128):
        assert call(K=K) == SHAPE
    assert call(rows=1 << 31) == SHAPE
    for arg in "abc":
        assert call(**{arg: None}) == INVALID
        assert call(**{arg: at(5, 8)}) == MISALIGNED
    assert call(c=at(0, 16)) == INVALID and call(c=at(1, 16)) == INVALID  # overlaps
    assert call(rows=0) == lg.LG_OK and call(a=None, rows=0) == lg.LG_OK


def test_linear_refusals():
    def call(x=at(0), xq=at(1), xs=at(2), wq=at(3), ws=at(4), A=at(5), B=at(6), y=at(7), M=10, K=256, N=64, R=64,
             work=at(8), nbytes=1 << 30):
        return L.lg_lora_linear_mxfp4(x, xq, xs, wq, ws, A, B, y, M, K, N, R, work, nbytes, None)

    assert call(M=-1) == INVALID
    for bad in (dict(K=64), dict(K=192), dict(N=40), dict(N=0), dict(R=32), dict(R=640), dict(M=1 << 31)):
        assert call(**bad) == SHAPE, bad
    for arg in ("x", "xq", "xs", "wq", "ws", "A", "B", "y"):
        assert call(**{arg: None}) == INVALID, arg
        assert call(**{arg: at(9, 4)}) == MISALIGNED, arg
    need = lg.lora_linear_mxfp4_workspace_size(10, 256, 64, 64)
    assert need > 0 and call(work=None) == WORKSPACE and call(nbytes=need - 1) == WORKSPACE
    assert call(work=at(8, 8)) == MISALIGNED
    for arg in ("x", "xq", "xs", "wq", "ws", "A", "B", "work"):
        assert call(y=at(9), **{arg: at(9)}) == INVALID, arg
    for arg in ("x", "xq", "xs", "wq", "ws", "A", "B"):
        assert call(work=at(9), **{arg: at(9)}) == INVALID, arg
    assert call(M=0) == lg.LG_OK
    assert call(M=0, R=0, x=None, A=None, B=None, work=None, nbytes=0) == lg.LG_OK
    for bad in ((10, 192, 64, 64), (10, 256, 48, 64), (10, 256, 64, 32), (-1, 256, 64, 64)):
        assert lg.lora_linear_mxfp4_workspace_size(*bad) == 0


def _norm(**kw):
    f = dict(h=at(0), b=at(1), gate=at(2), scale=at(3), shift=at(4), h_out=at(5), n=at(6), codes=at(7), scales=at(8),
             M=10, segment_tokens=4, D=256, stream_type=0, post=1, pre=1, codes_format=2, alpha=1.0, eps=1e-6)
    f.update(kw)
    return L.lg_block_norm(ctypes.byref(lg.BlockNormArgs(**f)), None)


def test_block_norm_refusals():
    assert L.lg_block_norm(None, None) == INVALID
    for bad in (dict(M=-1), dict(segment_tokens=0), dict(stream_type=2), dict(post=3), dict(pre=-1), dict(eps=0.0),
                dict(eps=-1.0), dict(eps=float("nan")), dict(alpha=float("inf")), dict(codes_format=3), dict(h=None),
                dict(codes=None), dict(scales=None), dict(codes_format=0), dict(h_out=None),
                dict(b=None), dict(b=None, h_out=None, post=0), dict(b=None, h_out=None, gate=None),
                dict(b=None, h_out=None, gate=None, post=0, alpha=0.5), dict(pre=0),
                dict(codes_format=0, codes=None, scales=None, n=None)):
        assert _norm(**bad) == INVALID, bad
    for bad in (dict(M=1 << 31), dict(D=0), dict(D=12), dict(D=264), dict(D=16512)):
        assert _norm(**bad) == SHAPE, bad
    for arg in ("h", "b", "gate", "scale", "shift", "h_out", "n", "codes", "scales"):
        assert _norm(**{arg: at(9, 8)}) == MISALIGNED, arg
    outs = ("h_out", "n", "codes", "scales")
    for i, out in enumerate(outs):
        for arg in ("h", "b", "gate", "scale", "shift") + outs[:i]:
            if (out, arg) != ("h_out", "h"):
                assert _norm(**{out: at(9), arg: at(9)}) == INVALID, (out, arg)
    assert _norm(h_out=at(0, 256)) == INVALID  # in place only as a whole
    assert _norm(M=0) == lg.LG_OK and _norm(M=0, h_out=at(0)) == lg.LG_OK
    assert _norm(M=0, pre=0, n=None, scale=None, shift=None, codes=None, scales=None, codes_format=0) == lg.LG_OK
    assert _norm(M=0, b=None, h_out=None, gate=None, post=0, n=None) == lg.LG_OK


def _back(work=at(20), nbytes=1 << 40, **kw):
    f = dict(dn=at(0), dh_out=at(1), h_out=at(2), b=at(3), gate=at(4), scale=at(5), dh=at(6), db=at(7), dgate=at(8),
             dscale=at(9), dshift=at(10), M=100, segment_tokens=50, D=256, stream_type=1, post=1, pre=1, alpha=1.0,
             eps=1e-6)
    f.update(kw)
    return L.lg_block_norm_backward(ctypes.byref(lg.BlockNormBackwardArgs(**f)), work, nbytes, None)


def test_block_norm_backward_refusals():
    assert L.lg_block_norm_backward(None, at(20), 1 << 40, None) == INVALID
    for bad in (dict(M=-1), dict(segment_tokens=0), dict(stream_type=7), dict(post=-1), dict(eps=0.0), dict(dn=None),
                dict(pre=0), dict(h_out=None), dict(b=None), dict(dn=None, pre=0),
                dict(dn=None, pre=0, scale=None, dscale=None), dict(dh=None, db=None, dgate=None, dscale=None, dshift=None)):
        assert _back(**bad) == INVALID, bad
    for bad in (dict(D=4), dict(D=20), dict(D=16392), dict(M=1 << 31)):
        assert _back(**bad) == SHAPE, bad
    for arg in ("dn", "dh_out", "h_out", "b", "gate", "scale", "dh", "db", "dgate", "dscale", "dshift", "work"):
        assert _back(**{arg: at(21, 4)}) == MISALIGNED, arg
    outs = ("dh", "db", "dgate", "dscale", "dshift", "work")
    for i, out in enumerate(outs):
        for arg in ("dn", "dh_out", "h_out", "b", "gate", "scale") + outs[:i]:
            if (out, arg) != ("dh", "dh_out"):
                assert _back(**{out: at(21), arg: at(21)}) == INVALID, (out, arg)
    need = lg.block_norm_backward_workspace_size(100, 256, 50)
    assert need > 0 and _back(nbytes=need - 1) == WORKSPACE and _back(work=None) == WORKSPACE
    # Segments of a chunk or less have no partial sums: no workspace.
    assert lg.block_norm_backward_workspace_size(100, 256, 1) == 0
    assert _back(M=0) == lg.LG_OK and _back(M=0, dh=at(1)) == lg.LG_OK
    for bad in ((0, 256, 4), (10, 12, 4), (10, 256, 0), (10, 1 << 20, 4)):
        assert lg.block_norm_backward_workspace_size(*bad) == 0


def test_binding_refusals():
    """The binding's own checks come before any pointer is taken (CPU tensors are refused as such)."""
    import torch

    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        lg.mxfp4_quantize(x)
    with pytest.raises(TypeError):
        lg.mxfp4_quantize(x.float())
    with pytest.raises(ValueError, match="CUDA"):
        lg.block_norm(x)
    with pytest.raises(TypeError):
        lg.block_norm(x.half())
    with pytest.raises(TypeError):
        lg.block_norm_backward(x, None, x.double())
