"""block_norm_backward where the parity tests of test_gpu_block_norm.py do not
reach.  Tolerances as there."""

import pytest
import torch

import lora_gemm_b200 as lg
from tests.test_gpu_block_norm import DEV, _check_backward, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [7168, 9216, 16384])
def test_a_row_s_meeting_is_bounded(D, stream):
    """Rows on clusters of two, four and eight CTAs: with a limit of a nanosecond the waits for the peers' sums
    give up, which is reported, and the device stays usable."""
    t = _inputs(600, D, 1, stream, seed=D)
    args = (t["dn"], t["dh"], t["h"], t["b"], t["gate"], t["scale"])
    want = lg.block_norm_backward(*args)
    assert lg.get_last_device_error() == lg.LG_OK
    lg.set_wait_limit_ns(1)
    try:
        lg.block_norm_backward(*args)
        assert lg.get_last_device_error() == lg.LG_ERR_DEVICE_TIMEOUT
    finally:
        lg.set_wait_limit_ns(0)
    got = lg.block_norm_backward(*args)
    assert lg.get_last_device_error() == lg.LG_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post", ["rms", "layer"])
@pytest.mark.parametrize("pre", ["rms", "layer"])
@pytest.mark.parametrize("size,eps", [(2.0 ** 50, 1e-6), (2.0 ** -50, 2.0 ** -110), (0.0, 1e-30)])
def test_rows_far_from_one(size, eps, pre, post, stream):
    """Reciprocal deviations of 2^-50, 2^50 and, rows of zeros, 1e15: their cubes are no FP32 numbers, the
    gradients are.  On one CTA and on a cluster, with the projection alone (no dh_out) and with a dh_out of
    its size."""
    for D in (1024, 4096):
        t = _inputs(5, D, 2, stream, seed=D)
        t["h"] *= size
        t["b"] *= size
        _check_backward(t, 5, D, 3, post, pre, 1.0, eps, dh_out=False)
        t["dh"] *= size ** -1 if size else eps ** -0.5
        got = _check_backward(t, 5, D, 3, post, pre, 1.0, eps)
        assert all(torch.isfinite(g).all() for g in got)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_without_norms_the_gradients_do_not_read_b(value):
    """h' = h + gate b: db = gate dh_out and dh = dh_out whatever b holds; dgate meets b in its own column alone."""
    t = _inputs(6, 512, 2, torch.float32, seed=11)
    b = t["b"].clone()
    b[4, 77] = value
    args = dict(post=None, pre=None, segment_tokens=3)
    dh, db, dgate, _, _ = lg.block_norm_backward(None, t["dh"], t["h"], b, t["gate"], **args)
    want = lg.block_norm_backward(None, t["dh"], t["h"], t["b"], t["gate"], **args)
    assert torch.equal(dh, want[0]) and torch.equal(db, want[1])
    assert torch.equal(db, (t["gate"].repeat_interleave(3, 0) * t["dh"]).to(torch.bfloat16))
    keep = torch.ones(2, 512, dtype=torch.bool, device=DEV)
    keep[1, 77] = False
    assert torch.equal(dgate[keep], want[2][keep]) and not torch.isfinite(dgate[1, 77])
