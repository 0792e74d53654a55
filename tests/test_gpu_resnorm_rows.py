"""lora_residual_norm_fwd and _bwd: a row's bits whatever the number of rows, and the stream's gradient in its own place."""
import pytest
import torch

import weight_patches_gb300 as wpg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dt,pad", [(BF, 4), (BF, 1), (F32, 2), (F32, 1)])
@pytest.mark.parametrize("C", [264, 1000, 4096])
def test_the_first_row_of_an_odd_pitch_has_the_bits_it_has_among_many(C, dt, pad):
    # the first row lies on 16 bytes, the others do not: whether it comes alone decides nothing
    g = torch.Generator(device=DEV).manual_seed(C + pad)
    mul = torch.randn(C, generator=g, device=DEV)
    for _ in range(8):
        x, y, dh = (torch.randn(5, C + pad, generator=g, device=DEV).to(dt)[:, :C] for _ in range(3))
        kw = dict(mul=mul, kind=wpg.WP_NORM_LAYER)
        for post in (None, wpg.WP_NORM_RMS):
            x1, h, st = wpg.lora_residual_norm_fwd(x, y, post_kind=post, **kw)
            b1, bh, bst = wpg.lora_residual_norm_fwd(x[:1], y[:1], post_kind=post, **kw)
            assert torch.equal(b1[0], x1[0]) and torch.equal(bh[0], h[0]) and torch.equal(bst[:2, 0], st[:2, 0])
            p = wpg.lora_residual_norm_bwd(dh, x, st, y, need_mul=False, post_kind=post, **kw)
            q = wpg.lora_residual_norm_bwd(dh[:1], x[:1], st[:, :1].contiguous(), y[:1], need_mul=False, post_kind=post, **kw)
            assert torch.equal(p.dX[0], q.dX[0]) and torch.equal(p.dY[0], q.dY[0])


@pytest.mark.parametrize("T,C,st,yt", [(40, 200, F32, BF), (900, 1536, F32, BF), (300, 1001, BF, BF), (64, 8192, F32, F32),
                                       (9, 16384, F32, F32)])
def test_the_streams_gradient_in_its_own_place(T, C, st, yt):
    g = torch.Generator(device=DEV).manual_seed(C)
    x, y, dh, dx1 = (torch.randn(T, C, generator=g, device=DEV).to(t) for t in (st, yt, yt, st))
    gate = torch.randn(C, generator=g, device=DEV)
    stats = wpg.lora_residual_norm_fwd(x, out_dtype=yt)[2]
    want = wpg.lora_residual_norm_bwd(dh, x, stats, y, dX1=dx1, gate=gate)
    # through the C entry: dX is dX1
    dy, dgate = torch.empty_like(dh), torch.empty(1, C, device=DEV)
    ws = torch.empty(wpg.lora_residual_norm_bwd_workspace_size(x), dtype=torch.uint8, device=DEV)
    a = wpg._residual_norm(gate, None, None, None, 1.0, 0.0, 0.0, 0.0, wpg.WP_NORM_LAYER, None)
    wpg._run(0, "lora_residual_norm_bwd", wpg._pmat(dh), wpg._pmat(dx1), wpg._pmat(x), wpg._pmat(y), stats.data_ptr(), a,
             wpg._pout(dx1), wpg._pout(dy), wpg._pout(dgate), None, None, None, ws.data_ptr(), ws.numel())
    assert torch.equal(dx1, want.dX) and torch.equal(dy, want.dY) and torch.equal(dgate[0], want.dgate)
