"""block_norm_backward where the parity tests of test_gpu_block_norm.py do not
reach.  Tolerances as there."""

import pytest
import torch

import lora_gemm_b200 as lg
from tests.test_gpu_block_norm import _inputs

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
