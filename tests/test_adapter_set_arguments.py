"""Arguments of the adapter-set calls that a kernel could not use: refused on the host, before any
pointer is passed on."""
import pytest
import torch

import weight_patches_gb300 as wpg

DEV = "cuda:0"


# ------------------------------------------------------------------------------ devices
def _calls(dev):
    """(call, its tensors by name) of every entry point that takes tensors, all on `dev`."""
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=dev)  # noqa: E731
    bf = torch.bfloat16

    def multi(X, W, bias, A, B, scale, slot, row_scale, out, workspace):
        bank = wpg.AdapterBank(A, B, scale)
        wpg.lora_linear_fwd_multi(X, W, bias, bank, slot, row_scale=row_scale, out=out, workspace=workspace)

    def multi_nf4(X, packed, absmax, A, B, scale, slot):
        wpg.lora_linear_fwd_multi(X, wpg.NF4Weight(packed, absmax, 32, 64), None, wpg.AdapterBank(A, B, scale), slot)

    def norm_fwd(X, weight, bias, out, stats):
        wpg.lora_norm_fwd(X, weight, bias, out=out, stats=stats)

    def norm_bwd(dY, X, weight, stats, workspace):
        wpg.lora_norm_bwd(dY, X, weight, stats, workspace=workspace)

    def adamw(p, m, v, g, scale):
        wpg.lora_adamw_step(wpg.lora_adamw_plan([p], [m], [v]), [g], 1e-3, grad_scale_tensor=scale)

    def decode(codes, absmax, out):
        wpg.lora_block8_decode(codes, absmax, out=out)

    bank = dict(A=z(2, 16, 64, dt=bf), B=z(2, 32, 16, dt=bf), scale=z(2), slot=z(3, dt=torch.int32))
    u8 = torch.uint8
    return {
        "multi": (multi, dict(bank, X=z(3, 64, dt=bf), W=z(32, 64, dt=bf), bias=z(32), row_scale=z(3),
                              out=z(3, 32, dt=bf), workspace=z(1 << 20, dt=u8))),
        "multi_nf4": (multi_nf4, dict(bank, X=z(3, 64, dt=bf), packed=z(32, 32, dt=u8), absmax=z(32))),
        "norm_fwd": (norm_fwd, dict(X=z(3, 64), weight=z(64), bias=z(64), out=z(3, 64), stats=z(2, 3))),
        "norm_bwd": (norm_bwd, dict(dY=z(3, 64), X=z(3, 64), weight=z(64), stats=z(2, 3), workspace=z(1 << 20, dt=u8))),
        "adamw": (adamw, dict(p=z(300), m=z(300), v=z(300), g=z(300), scale=z(1))),
        "decode": (decode, dict(codes=z(300, dt=u8), absmax=z(2), out=z(300))),
    }


@pytest.mark.parametrize("name", list(_calls("cpu")))
def test_host_tensors_are_refused(name):
    call, tensors = _calls("cpu")[name]
    with pytest.raises(ValueError, match="device"):
        call(**tensors)


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(_calls("cpu")))
def test_one_tensor_on_the_host_is_refused(name):
    call, tensors = _calls(DEV)[name]
    call(**tensors)
    for k in tensors:
        with pytest.raises(ValueError, match="device"):
            call(**{**tensors, k: tensors[k].cpu()})
    torch.cuda.synchronize()
    assert wpg.lora_device_status() == 0
