"""GPU parity of block_norm and block_norm_backward with the FP64 oracle.

Tolerances.  A rounding to the output type costs half a step: eps / 2 of the
value (bf16 2^-8, FP32 2^-24).  Statistics are FP32 sums of at most 32 terms
per thread and a tree over the threads: below 64 roundings, 64 x 2^-24 = 2^-18
of the sum of magnitudes; a reciprocal deviation takes half of that.  An output
is therefore held to half a step plus 2^-16 of the magnitudes that enter it
(four such errors).  Column sums add up to `rows` roundings."""

import numpy as np
import pytest
import torch

import lora_gemm_b200 as lg
from oracle import mxfp4 as o4
from oracle import norm as on

pytestmark = pytest.mark.gpu
DEV = "cuda"
FP = 2.0 ** -16
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _np64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def _inputs(M, D, S, stream, seed, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    t = {"h": (torch.randn(M, D, generator=g) * torch.exp2(torch.randn(M, 1, generator=g)) + mean).to(stream),
         "b": (torch.randn(M, D, generator=g) + mean).to(torch.bfloat16),
         "gate": torch.randn(S, D, generator=g) * 0.5, "scale": torch.randn(S, D, generator=g) * 0.3,
         "shift": torch.randn(S, D, generator=g) * 0.3, "dn": torch.randn(M, D, generator=g).to(torch.bfloat16),
         "dh": torch.randn(M, D, generator=g).to(stream)}
    return {k: v.to(DEV) for k, v in t.items()}


def _near(got, want, tol, what):
    bad = ~(np.abs(_np64(got) - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist())


def _check_forward(t, M, D, seg, post, pre, alpha, eps, **kw):
    """h' against the formula, n against the formula on the h' that came back."""
    has_b = kw.pop("has_b", True)
    a = {k: _np64(v) for k, v in t.items()}
    stream = t["h"].dtype
    args = dict(alpha=alpha, eps=eps, post=post, pre=pre, segment_tokens=seg)
    h_in = t["h"].clone()
    h, n, q = lg.block_norm(t["h"], t["b"] if has_b else None, t["gate"] if has_b else None,
                            t["scale"] if pre else None, t["shift"] if pre else None, **args, **kw)
    if has_b:
        u, r = on.normalise(a["b"], post, eps)
        gate = np.abs(on.rows_of(a["gate"], M, seg, 1.0))
        off = 0.0 if post is None else np.abs(u) + r * np.abs(a["b"]).mean(1, keepdims=True) * (post == "layer")
        want = on.residual(_np64(h_in), a["b"], a["gate"], alpha, eps, post, seg)
        _near(h, want, STEP[stream] * np.abs(want) + FP * (np.abs(alpha * _np64(h_in)) + gate * (np.abs(u) + off)), "h")
    else:
        assert h is t["h"] and torch.equal(h, h_in)
    if pre is None:
        assert n is None
        return h, n, q
    ho = _np64(h)
    x, r = on.normalise(ho, pre, eps)
    mul = np.abs(1.0 + on.rows_of(a["scale"], M, seg, 0.0))
    mag = np.abs(x) + r * np.abs(ho).mean(1, keepdims=True) * (pre == "layer")
    want = on.modulated(ho, a["scale"], a["shift"], eps, pre, seg)
    if n is not None:
        _near(n, want, 2.0 ** -8 * np.abs(want) + FP * (mag * mul + np.abs(on.rows_of(a["shift"], M, seg, 0.0))), "n")
    return h, n, q


SHAPES = [(1, 8, 1), (3, 64, 2), (5, 248, 5), (130, 256, 40), (33, 512, 7), (40, 1000, 13), (9, 1024, 100), (7, 1032, 3),
          (6, 7168, 4), (5, 8192, 2), (3, 9000, 2), (2, 16384, 1)]


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,D,seg", SHAPES)
def test_forward_shapes(M, D, seg, stream):
    t = _inputs(M, D, -(-M // seg), stream, seed=M * D)
    _check_forward(t, M, D, seg, "rms", "layer", 0.7, 1e-5)


@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("pre", [None, "rms", "layer"])
@pytest.mark.parametrize("D", [256, 2048])
def test_forward_kinds(post, pre, D):
    t = _inputs(23, D, 3, torch.float32, seed=D)
    _check_forward(t, 23, D, 10, post, pre, 1.0, 1e-6)


@pytest.mark.parametrize("pre", ["rms", "layer"])
def test_forward_without_block_output_or_modulation(pre):
    t = _inputs(9, 640, 1, torch.bfloat16, seed=1)
    _check_forward(t, 9, 640, 9, None, pre, 1.0, 1e-6, has_b=False)
    h, n, _ = lg.block_norm(t["h"], pre=pre)
    want = on.normalise(_np64(t["h"]), pre, 1e-6)[0]
    _near(n, want, 2.0 ** -8 * np.abs(want) + 8 * FP, "n")


def test_layer_norm_of_rows_far_from_zero():
    """A mean 300 times the deviation: the squares must be those of centred values."""
    t = _inputs(11, 2048, 1, torch.float32, seed=5, mean=300.0)
    _check_forward(t, 11, 2048, 11, "layer", "layer", 1.0, 1e-6)


def test_rows_of_zeros_and_of_one_value():
    t = _inputs(4, 512, 1, torch.float32, seed=6)
    t["h"][0], t["b"][0] = 0.0, 0.0
    t["h"][1], t["b"][1] = 3.0, 3.0
    for kind in ("rms", "layer"):
        h, n, _ = _check_forward(t, 4, 512, 4, kind, kind, 1.0, 1e-6)
        assert torch.isfinite(h).all() and torch.isfinite(n).all()


def test_nan_stays_in_its_row():
    t = _inputs(6, 1536, 1, torch.bfloat16, seed=8)
    t["b"][2, 700] = float("nan")
    t["h"][4, 3] = float("inf")
    h, n, q = lg.block_norm(t["h"], t["b"], quant="mxfp4")
    bad = torch.isnan(n).any(1).cpu()
    assert bad.tolist() == [False, False, True, False, True, False]
    v = lg.mxfp4_dequantize(*q)
    assert torch.isnan(v[2]).all() and torch.isfinite(v[[0, 1, 3, 5]]).all()


@pytest.mark.parametrize("M,D", [(1, 128), (130, 256), (37, 1024), (129, 7168), (5, 16384)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_codes_are_the_quantizers(M, D, stream):
    """The fused codes equal the quantizers' of the returned n, bit for bit, padding rows included."""
    t = _inputs(M, D, 1, stream, seed=M + D)
    for quant, fn in (("mxfp4", lg.mxfp4_quantize), ("mxfp8", lg.mx_quantize)):
        _, n, q = lg.block_norm(t["h"], t["b"], t["gate"], t["scale"], t["shift"], quant=quant)
        want = fn(n)
        assert torch.equal(q[0], want[0]) and torch.equal(q[1], want[1][:q[1].numel()]), quant
    c, s = o4.mx_quantize(_np64(lg.block_norm(t["h"])[1]))
    got, _ = lg.block_norm(t["h"], quant="mxfp4")[2]
    assert np.array_equal(got.cpu().numpy(), o4.pack(c))


def test_in_place_and_neighbours():
    """h_out may be h; rows behind the last token and bytes behind the scales are left alone."""
    t = _inputs(10, 768, 2, torch.bfloat16, seed=4)
    want = lg.block_norm(t["h"], t["b"], t["gate"], t["scale"], t["shift"], segment_tokens=6)
    buf = torch.full((14, 768), 5.0, dtype=torch.bfloat16, device=DEV)
    buf[:10] = t["h"]
    nb = torch.full((14, 768), 5.0, dtype=torch.bfloat16, device=DEV)
    h, n, _ = lg.block_norm(buf[:10], t["b"], t["gate"], t["scale"], t["shift"], segment_tokens=6, h_out=buf[:10],
                            n=nb[:10])
    assert torch.equal(h, want[0]) and torch.equal(n, want[1]) and h.data_ptr() == buf.data_ptr()
    assert (buf[10:] == 5.0).all() and (nb[10:] == 5.0).all()


def _shifted(t, by):
    """The same values at an address `by` elements past a 512-byte boundary."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)
    out = buf[by:].view_as(t)
    out.copy_(t)
    return out


def test_addresses_aligned_to_16_bytes_only():
    """FP32 rows and modulations 16 bytes off a 32-byte boundary: same bits as aligned ones."""
    t = _inputs(12, 520, 2, torch.float32, seed=21)
    s = {k: _shifted(v, 4 if v.dtype == torch.float32 else 8) for k, v in t.items()}
    for x, y in zip(lg.block_norm(t["h"], t["b"], t["gate"], t["scale"], t["shift"], segment_tokens=7)[:2],
                    lg.block_norm(s["h"], s["b"], s["gate"], s["scale"], s["shift"], segment_tokens=7,
                                  h_out=_shifted(t["h"], 4))[:2]):
        assert torch.equal(x, y)
    a = lg.block_norm_backward(t["dn"], t["dh"], t["h"], t["b"], t["gate"], t["scale"], segment_tokens=7)
    b = lg.block_norm_backward(s["dn"], s["dh"], s["h"], s["b"], s["gate"], s["scale"], segment_tokens=7, dh=s["dh"])
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def _check_backward(t, M, D, seg, post, pre, alpha, eps, has_b=True, dh_out=True):
    a = {k: _np64(v) for k, v in t.items()}
    stream = t["h"].dtype
    got = lg.block_norm_backward(t["dn"] if pre else None, t["dh"] if dh_out else None, t["h"],
                                 t["b"] if has_b else None, t["gate"] if has_b else None, t["scale"] if pre else None,
                                 alpha=alpha, eps=eps, post=post, pre=pre, segment_tokens=seg)
    want = on.backward(a["dn"] if pre else None, a["dh"] if dh_out else None, a["h"], a["b"] if has_b else None,
                       a["gate"] if has_b else None, a["scale"] if pre else None, alpha, eps, post, pre, seg)
    rows = min(seg, M) + 64
    mag = np.abs(a["dh"]) if dh_out else np.zeros((M, D))
    if pre:
        x, r = on.normalise(a["h"], pre, eps)
        x = np.abs(x) + r * np.abs(a["h"]).mean(1, keepdims=True) * (pre == "layer")
        g = np.abs(a["dn"] * (1.0 + on.rows_of(a["scale"], M, seg, 0.0)))
        mag = mag + r * (g + g.mean(1, keepdims=True) + x * (g * x).mean(1, keepdims=True))
        _near(got[3], want[3], (FP + rows * 2.0 ** -24) * on.segment_sums(np.abs(a["dn"]) * x, seg), "dscale")
        _near(got[4], want[4], rows * 2.0 ** -24 * on.segment_sums(np.abs(a["dn"]), seg), "dshift")
    else:
        assert got[3] is None and got[4] is None
    _near(got[0], want[0], STEP[stream] * np.abs(want[0]) + FP * abs(alpha) * mag, "dh")
    if has_b:
        u, r = on.normalise(a["b"], post, eps)
        w = np.abs(on.rows_of(a["gate"], M, seg, 1.0)) * mag
        if post is None:
            tol = FP * w
        else:
            u = np.abs(u) + r * np.abs(a["b"]).mean(1, keepdims=True) * (post == "layer")
            tol = 2 * FP * r * (w + w.mean(1, keepdims=True) + u * (w * u).mean(1, keepdims=True))
        _near(got[1], want[1], 2.0 ** -8 * np.abs(want[1]) + tol, "db")
        _near(got[2], want[2], (2 * FP + rows * 2.0 ** -24) * on.segment_sums(mag * np.abs(u), seg), "dgate")
    else:
        assert got[1] is None and got[2] is None
    return got


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,D,seg", SHAPES + [(700, 64, 700), (300, 1024, 1), (513, 2048, 200), (150, 8200, 149)])
def test_backward_shapes(M, D, seg, stream):
    t = _inputs(M, D, -(-M // seg), stream, seed=M * D + 1)
    _check_backward(t, M, D, seg, "layer", "rms", 0.7, 1e-5)


@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("pre", [None, "rms", "layer"])
def test_backward_kinds(post, pre):
    t = _inputs(90, 1280, 2, torch.float32, seed=9)
    _check_backward(t, 90, 1280, 70, post, pre, 1.0, 1e-6)


def test_backward_without_block_output_and_without_stream_gradient():
    t = _inputs(20, 640, 1, torch.bfloat16, seed=2)
    _check_backward(t, 20, 640, 20, None, "rms", 1.0, 1e-6, has_b=False)
    _check_backward(t, 20, 640, 20, "rms", "layer", 1.0, 1e-6, dh_out=False)


def test_backward_repeats_bit_for_bit_and_in_place():
    t = _inputs(1000, 512, 3, torch.bfloat16, seed=3)
    args = dict(segment_tokens=400)
    one = lg.block_norm_backward(t["dn"], t["dh"], t["h"], t["b"], t["gate"], t["scale"], **args)
    dh = t["dh"].clone()
    two = lg.block_norm_backward(t["dn"], dh, t["h"], t["b"], t["gate"], t["scale"], dh=dh, **args)
    assert all(torch.equal(a, b) for a, b in zip(one, two)) and two[0].data_ptr() == dh.data_ptr()


def test_gradients_against_differences_of_the_kernel():
    """Directional derivative of an FP32-stream call: central differences of the
    kernel's own h' (n is rounded to bf16: its part is taken from FP64).  The
    step 2^-6 leaves a truncation of order 2^-12 and FP32 noise of 2^-24 x 2^6."""
    M, D, seg = 6, 512, 3
    t = _inputs(M, D, 2, torch.float32, seed=12)
    _, db, dgate, _, _ = lg.block_norm_backward(None, t["dh"], t["h"], t["b"], t["gate"], post="rms", pre=None,
                                                segment_tokens=seg)
    v = torch.randn(2, D, generator=torch.Generator().manual_seed(1)).to(DEV)

    def loss(gate):
        h, _, _ = lg.block_norm(t["h"], t["b"], gate, post="rms", pre=None, segment_tokens=seg)
        return float((h.double() * t["dh"].double()).sum())

    num = (loss(t["gate"] + 2.0 ** -6 * v) - loss(t["gate"] - 2.0 ** -6 * v)) / 2.0 ** -5
    want = float((dgate.double() * v.double()).sum())
    size = float((dgate.double() * v.double()).norm())
    assert abs(num - want) <= 1e-3 * size
