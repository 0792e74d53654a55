"""The residual norm's bounded waits, made to run out on purpose: under lora_debug_hold_flags no row is sent for, so that each
CTA's first wait expires.  Whole warps leave, the status word says so, and the next calls on the device are right."""
import time

import pytest
import torch

import weight_patches_gb300 as wpg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T,C,post", [(700, 1536, None), (40, 4096, wpg.WP_NORM_RMS), (33, 1001, None), (3, 8192, wpg.WP_NORM_LAYER)])
def test_a_wait_that_runs_out_leaves_the_device_usable(T, C, post):
    g = torch.Generator(device=DEV).manual_seed(C)
    x, y, dh = (torch.randn(T, C, generator=g, device=DEV).bfloat16() for _ in range(3))
    gate = torch.randn(C, generator=g, device=DEV)
    fwd = lambda: wpg.lora_residual_norm_fwd(x, y, gate=gate, post_kind=post)  # noqa: E731
    x1, h, stats = fwd()
    bwd = lambda: wpg.lora_residual_norm_bwd(dh, x1, stats, y, gate=gate, post_kind=post)  # noqa: E731
    grads = bwd()
    torch.cuda.synchronize()
    for call in (fwd, bwd):
        assert wpg.lora_device_status(reset=True) in (0, -7)       # start clean
        wpg.lora_set_wait_limit(50_000_000)
        wpg.lib().lora_debug_hold_flags(1)
        try:
            t0 = time.time()
            call()
            torch.cuda.synchronize()
            elapsed = time.time() - t0
            assert wpg.lora_device_status(reset=True) == -7
        finally:
            wpg.lib().lora_debug_hold_flags(0)
            wpg.lora_set_wait_limit(2_000_000_000)
        assert elapsed < 30.0, elapsed
    again = fwd()
    assert torch.equal(again[0], x1) and torch.equal(again[1], h)
    for a, b in zip(bwd(), grads):
        assert a is None and b is None or torch.equal(a, b)
    torch.cuda.synchronize()
    assert wpg.lora_device_status() == 0
