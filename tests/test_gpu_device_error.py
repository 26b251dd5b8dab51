"""What get_last_device_error costs: one copy from the device for each family of
kernels with bounded waits that the process has launched, and none for the others."""

import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

SCRIPT = textwrap.dedent("""
    import torch
    from torch.profiler import ProfilerActivity, profile
    import lora_gemm_b200 as lg

    def copies():
        with profile(activities=[ProfilerActivity.CUDA]) as p:
            assert lg.get_last_device_error() == lg.LG_OK
            torch.cuda.synchronize()
        return sum("Memcpy DtoH" in e.name for e in p.events())

    x = torch.randn(200, 256, device="cuda").bfloat16()
    W = torch.randn(64, 256, device="cuda").bfloat16()
    q, Wq = lg.mxfp4_quantize(x), lg.mxfp4_quantize(W)
    t = torch.randn(3, 4096, device="cuda").bfloat16()
    counts = []
    for call in (lambda: lg.lora_linear(x, W, None, None),
                 lambda: lg.block_norm_backward(t[:, :256].contiguous(), None, t[:, :256].contiguous()),  # no wait
                 lambda: lg.lora_linear_mxfp4(None, q, Wq, None, None),
                 lambda: lg.lora_linear_mxfp4(None, lg.mxfp4_quantize(x[:5]), Wq, None, None),
                 lambda: lg.block_norm_backward(t, None, t),
                 lambda: lg.lora_linear(x, W, None, None)):
        call()
        counts.append(copies())
    print("copies", *counts)
""")


def test_copies_of_the_error_words():
    out = subprocess.run([sys.executable, "-c", SCRIPT], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr[-2000:]
    assert "copies 1 1 2 3 4 4" in out.stdout, out.stdout
