"""lora_ce_bwd of padded batches: rows that do not count change nothing of the other rows' gradients."""
import pytest
import torch

import weight_patches_gb300 as wpg
from tests.test_gpu_ce import DEV, case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,n", [(513, 512), (600, 40), (1500, 500), (9000, 1), (700, 320)])
def test_rows_that_do_not_count_leave_dw_as_it_is(T, n):
    # dW's terms are rounded by the rows that count, not by the rows that were passed: a padded batch has the bits of
    # the rows alone
    x, w, y = case(n, 136, 700, seed=T)
    lse = wpg.lora_ce_fwd(x, w, y)[1]
    d = torch.rand(n, device=DEV) + 0.5
    at = torch.randperm(T, generator=torch.Generator().manual_seed(T))[:n].sort().values.to(DEV)
    wide = torch.randn(T, 136, device=DEV).bfloat16()
    wide[at] = x
    yw = torch.full((T,), -100, device=DEV)
    lw, dw = torch.zeros(T, device=DEV), torch.ones(T, device=DEV)
    yw[at], lw[at], dw[at] = y, lse, d
    for dt in (torch.float32, torch.bfloat16):
        want = wpg.lora_ce_bwd(x, w, y, lse, d, need_dX=False, dW_dtype=dt)[1]
        ws = torch.full((wpg.lora_ce_workspace_size(wide, w, True),), 255, dtype=torch.uint8, device=DEV)      # NaN
        got = wpg.lora_ce_bwd(wide, w, yw, lw, dw, need_dX=False, dW_dtype=dt, workspace=ws)[1]
        assert torch.equal(got, want)
    torch.cuda.synchronize()
    assert wpg.lora_device_status() == 0


def test_one_row_of_a_short_pitch():
    # the transpose of a column: strides (1, 1)
    x, w, y = case(1, 512, 40)
    col = torch.empty(512, 1, dtype=torch.bfloat16, device=DEV).t()
    col.copy_(x)
    assert col.stride() == (1, 1)
    d = torch.ones(1, device=DEV)
    a, b = wpg.lora_ce_fwd(x, w, y), wpg.lora_ce_fwd(col, w, y)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = wpg.lora_ce_bwd(x, w, y, a[1], d), wpg.lora_ce_bwd(col, w, y, a[1], d)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
