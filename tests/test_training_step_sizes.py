"""Workspace sizes of the operators around the adapted linears are those of the calls, whatever pitch a matrix of one row or
one column comes with (host only: no GPU needed)."""
import ctypes

import pytest
import torch

import weight_patches_gb300 as wpg

BF = torch.bfloat16


def one_row(K):
    t = torch.zeros(K, 1, dtype=BF).t()
    assert t.stride() == (1, 1)
    return t


@pytest.mark.parametrize("backward", [False, True])
def test_ce_one_row_of_a_short_pitch(backward):
    K = 512
    x, w = torch.zeros(1, K, dtype=BF), torch.zeros(9, K, dtype=BF)
    want = wpg.lora_ce_workspace_size(x, w, backward)
    assert want > 0 and wpg.lora_ce_workspace_size(one_row(K), w, backward) == want
    want = wpg.lora_ce_workspace_size(w, x, backward)
    assert want > 0 and wpg.lora_ce_workspace_size(w, one_row(K), backward) == want


@pytest.mark.parametrize("ld", [0, 1, 63, 64, 65, 1 << 40])
def test_the_library_takes_one_row_of_any_pitch(ld):
    mat = lambda rows, ld: ctypes.byref(wpg.WpMat(0x10000, wpg.WP_BF16, rows, 64, ld, None))  # noqa: E731
    size = wpg.lib().lora_ce_workspace_size
    for b in (0, 1):
        assert size(mat(1, ld), mat(9, 64), b) == size(mat(1, 64), mat(9, 64), b) > 0
        assert size(mat(9, 64), mat(1, ld), b) == size(mat(9, 64), mat(1, 64), b) > 0
        assert (size(mat(2, ld), mat(9, 64), b) > 0) == (ld >= 64 and ld % 8 == 0)


def test_residual_norm_rows_of_one_column():
    x = torch.zeros(1, 5).t()                                   # [5, 1], strides (1, 5)
    assert wpg.lora_residual_norm_bwd_workspace_size(x) == wpg.lora_residual_norm_bwd_workspace_size(x.contiguous()) > 0
