"""The new operators run together, as a step runs them: norm -> 4-bit linear ->
norm, eager and captured, on other streams, two at a time, and backward; and the
shared failure path (bounded waits)."""

import numpy as np
import pytest
import torch

import lora_gemm_b200 as lg
from oracle import mxfp4 as o4
from oracle import norm as on
from tests.util import rel_fro

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _setup(M, D, N, R, seg, seed):
    g = torch.Generator().manual_seed(seed)
    S = -(-M // seg)
    t = {"h": torch.randn(M, D, generator=g).to(torch.bfloat16), "b": torch.randn(M, D, generator=g).to(torch.bfloat16),
         "gate": torch.randn(S, D, generator=g) * 0.3, "scale": torch.randn(S, D, generator=g) * 0.2,
         "shift": torch.randn(S, D, generator=g) * 0.2, "A": torch.randn(R, D, generator=g) * D ** -0.5,
         "B": torch.randn(N, R, generator=g) * 0.05}
    t = {k: v.to(DEV) for k, v in t.items()}
    W = (torch.randn(N, D, generator=g) * D ** -0.5).to(torch.bfloat16).to(DEV)
    t["W"] = lg.mxfp4_quantize(W)
    t["W16"] = W
    return t


def _block(t, seg):
    """One block: norm with 4-bit hand-over, the linear, and the norm after it."""
    h, n, q = lg.block_norm(t["h"], t["b"], t["gate"], t["scale"], t["shift"], alpha=0.7, segment_tokens=seg,
                            quant="mxfp4")
    y = lg.lora_linear_mxfp4(n, q, t["W"], t["A"], t["B"])
    return (h, n, q[0], q[1], y) + lg.block_norm(h, y, t["gate"], alpha=0.7, segment_tokens=seg, pre="layer")[:2]


@pytest.mark.parametrize("M", [3, 90, 300])
def test_block_against_the_oracle(M):
    D, R, seg = 512, 128, 50
    t = _setup(M, D, D, R, seg, seed=M)
    h, n, _, _, y, h2, n2 = _block(t, seg)
    a = {k: _np64(t[k]) for k in ("h", "b", "gate", "scale", "shift", "A", "B")}
    want_h = on.residual(a["h"], a["b"], a["gate"], 0.7, 1e-6, "rms", seg)
    assert rel_fro(_np64(h), want_h) <= 2.0 ** -8
    assert rel_fro(_np64(n), on.modulated(_np64(h), a["scale"], a["shift"], 1e-6, "rms", seg)) <= 2.0 ** -8
    ref = o4.lora_linear_mxfp4(_np64(n), _np64(t["W16"]), a["A"], a["B"])
    assert rel_fro(_np64(y), ref) <= 1e-2
    want_h2 = on.residual(_np64(h), _np64(y), a["gate"], 0.7, 1e-6, "rms", seg)
    assert rel_fro(_np64(h2), want_h2) <= 2.0 ** -8
    assert rel_fro(_np64(n2), on.modulated(_np64(h2), None, None, 1e-6, "layer", seg)) <= 2.0 ** -8


@pytest.mark.parametrize("M", [1, 77, 200, 700])
def test_captured_block_replays(M):
    """Captured once, replayed on new inputs: the bits of the eager calls."""
    D, seg = 512, 64
    t = _setup(M, D, D, 64, seg, seed=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _block(t, seg)
        lg.block_norm_backward(t["b"], t["h"], t["h"], t["b"], t["gate"], t["scale"], segment_tokens=seg)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = _block(t, seg)
        back = lg.block_norm_backward(t["b"], t["h"], t["h"], t["b"], t["gate"], t["scale"], segment_tokens=seg)
    for seed in (2, 3):
        new = _setup(M, D, D, 64, seg, seed)
        for k in ("h", "b", "gate", "scale", "shift", "A", "B"):
            t[k].copy_(new[k])
        t["W"][0].copy_(new["W"][0])
        t["W"][1].copy_(new["W"][1])
        g.replay()
        torch.cuda.synchronize()
        want = _block(new, seg)
        wback = lg.block_norm_backward(new["b"], new["h"], new["h"], new["b"], new["gate"], new["scale"], segment_tokens=seg)
        assert all(torch.equal(x, w) for x, w in zip(out, want))
        assert all(torch.equal(x, w) for x, w in zip(back, wback))
    assert lg.get_last_device_error() == lg.LG_OK


def test_two_streams_at_once():
    """Blocks of three sizes on two streams, many at a time, each with its own workspaces: the bits of one alone."""
    cases = [(5, 1024), (100, 512), (400, 512)]
    sets = [_setup(M, D, D, 64, 64, seed=M) for M, D in cases]
    want = [_block(t, 64) for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for k in range(12):
        with torch.cuda.stream(streams[k % 2]):
            got.append((k % 3, _block(sets[k % 3], 64)))
    torch.cuda.synchronize()
    for i, out in got:
        assert all(torch.equal(x, w) for x, w in zip(out, want[i]))
    assert lg.get_last_device_error() == lg.LG_OK


@pytest.mark.parametrize("M", [2, 100, 300])
def test_linear_calls_back_to_back_share_a_workspace(M):
    """Ordered calls on one stream may share a workspace: a call's first kernel waits for the call before."""
    t = _setup(M, 1024, 768, 576, 64, seed=5)
    x1, x2 = t["h"], t["b"]
    q1, q2 = lg.mxfp4_quantize(x1), lg.mxfp4_quantize(x2)
    want = [lg.lora_linear_mxfp4(x, q, t["W"], t["A"], t["B"]) for x, q in ((x1, q1), (x2, q2))]
    ws = torch.empty(lg.lora_linear_mxfp4_workspace_size(M, 1024, 768, 576), dtype=torch.uint8, device=DEV)
    for _ in range(20):
        got = [lg.lora_linear_mxfp4(x, q, t["W"], t["A"], t["B"], workspace=ws) for x, q in ((x1, q1), (x2, q2))]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_padded_batch():
    """A batch padded with zero rows: the live rows' bits do not depend on the padding, and zero rows stay finite."""
    t = _setup(150, 512, 512, 64, 150, seed=9)
    one = _block(t, 150)
    pad = dict(t)
    for k in ("h", "b"):
        pad[k] = torch.cat([t[k], torch.zeros(61, 512, dtype=torch.bfloat16, device=DEV)])
    two = _block(pad, 211)
    for i in (0, 1, 2, 4, 5, 6):
        assert torch.equal(one[i], two[i][:150])
        assert i == 2 or torch.isfinite(two[i][150:]).all()


def test_waits_are_bounded():
    """With a limit of a nanosecond the pipelined kernels give up, report it and leave the device usable."""
    t = _setup(100, 7168, 256, 64, 100, seed=4)
    q = lg.mxfp4_quantize(t["h"])
    want = lg.lora_linear_mxfp4(t["h"], q, t["W"], t["A"], t["B"])
    lg.set_wait_limit_ns(1)
    try:
        lg.lora_linear_mxfp4(t["h"], q, t["W"], t["A"], t["B"])
        assert lg.get_last_device_error() == lg.LG_ERR_DEVICE_TIMEOUT
    finally:
        lg.set_wait_limit_ns(0)
    assert lg.get_last_device_error() == lg.LG_OK
    assert torch.equal(lg.lora_linear_mxfp4(t["h"], q, t["W"], t["A"], t["B"]), want)


def test_long_offsets():
    """Tensors past 2^31 elements and 2^32 bytes: the last rows are computed like the same rows alone."""
    M, D = 305_000, 7168
    x = torch.zeros(M, D, dtype=torch.bfloat16, device=DEV)
    tail = torch.randn(70, D, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).to(DEV)
    x[-70:] = tail
    codes, scales = lg.mxfp4_quantize(x)
    alone = lg.mxfp4_quantize(tail)
    assert torch.equal(codes[-70:], alone[0])
    v = lg.mxfp4_dequantize(codes, scales)
    assert torch.equal(v[-70:], lg.mxfp4_dequantize(*alone)) and not v[: M - 70].any()
    del v
    gate = torch.randn(1, D, generator=torch.Generator().manual_seed(1)).to(DEV)
    with pytest.raises(lg.LoraGemmError):
        lg.block_norm(x, x, gate, h_out=x)  # in place is for the stream, not for b
    h, n, q = lg.block_norm(x, x.clone(), gate, quant="mxfp4", h_out=x)
    want = lg.block_norm(tail, tail, gate, quant="mxfp4")
    assert torch.equal(h[-70:], want[0]) and torch.equal(n[-70:], want[1]) and torch.equal(q[0][-70:], want[2][0])
    W = lg.mxfp4_quantize(torch.randn(256, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV))
    y = lg.lora_linear_mxfp4(n, q, W, None, None)
    tail_q = lg.mxfp4_quantize(n[-300:].contiguous())
    assert torch.equal(y[-300:], lg.lora_linear_mxfp4(None, tail_q, W, None, None))
    del q, y, codes
    dh, db, dgate, dscale, dshift = lg.block_norm_backward(n, None, h, n, gate)
    one = lg.block_norm_backward(n[-70:], None, h[-70:], n[-70:], gate)
    assert torch.equal(dh[-70:], one[0]) and torch.equal(db[-70:], one[1])
    torch.cuda.empty_cache()
