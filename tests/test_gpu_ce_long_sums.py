"""lora_ce_bwd where a sum is long: contractions over many columns, vocabulary entries and rows.

The tensor core adds 16 products a step to its accumulator and cuts the sum: by at most 17 units of 2^-23 of the magnitudes
that meet there, 2.125 of 2^-24 a product.  The kernels do so over 4096 products at most and add such chunks with
rounding to nearest, so that a sum of n products is within (2.125 min(n, 4096) + n / 4096 + 4) units of 2^-24 of its terms'
magnitudes."""
import numpy as np
import pytest
import torch

import weight_patches_gb300 as wpg
from tests.test_gpu_ce import DEV, U16, U32, case

pytestmark = pytest.mark.gpu


def units(n):
    return (2.125 * min(n, 4096) + n / 4096 + 4) * U32


# ---------------------------------------------------------------------------- several chunks of K
@pytest.mark.parametrize("T,K,V", [(300, 1032, 700), (64, 2056, 513), (257, 4104, 1000), (520, 1536, 300), (5000, 8200, 300)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_backward(T, K, V, dt):
    x, w, y = case(T, K, V, seed=T + K, ignored=0.1)
    keep = (y >= 0) & (y < V)
    rows = keep.nonzero()[:, 0]
    xd, wd, n = x[rows].double(), w.double(), len(rows)
    z = xd @ wd.t()
    lse = torch.zeros(T, device=DEV)
    lse[rows] = torch.logsumexp(z, 1).float()
    d = torch.rand(T, device=DEV) * 2 - 0.5
    dx, dw = wpg.lora_ce_bwd(x, w, y, lse, d, dX_dtype=dt, dW_dtype=dt)
    torch.cuda.synchronize()
    assert wpg.lora_device_status() == 0
    hot = torch.nn.functional.one_hot(y[rows], V).double()
    G = (torch.exp(z - lse[rows].double()[:, None]) - hot) * d[rows].double()[:, None]
    # one bf16 rounding, the logit's error, the exponential and the base-2 logit's roundings (2^-18, as in test_gpu_ce)
    p = G.abs() + 2 * d[rows].double().abs()[:, None] * hot
    dG = U16 * G.abs() * (1 + U16) + 1.01 * p * (units(K) * (xd.abs() @ wd.abs().t()) + 2.0 ** -18)
    out = U16 if dt == torch.bfloat16 else U32
    want = G @ wd
    err = dG @ wd.abs() + units(V) * (G.abs() @ wd.abs())
    assert bool(((dx[rows].double() - want).abs() <= err * (1 + out) + out * want.abs()).all())
    assert bool((dx[~keep] == 0).all())
    # X times the row's factor: in two bf16 parts, or one
    dG = dG + (2.0 ** -16 if n <= 512 else U16 * (1 + U16)) * G.abs()
    want = G.t() @ xd
    err = dG.t() @ xd.abs() + units(2 * n) * (G.abs().t() @ xd.abs())
    assert bool(((dw.double() - want).abs() <= err * (1 + out) + out * want.abs()).all())


# ------------------------------------------------------------------------------------ long sums
# All terms are positive and alike, so that cuts add up in one direction.
def test_backward_of_very_long_rows():
    # W's last V columns are one-hot and X has zeros there, so that dX in fp32 shows G's entries in these columns
    T, V, K0 = 64, 64, 1 << 20
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.zeros(T, K0 + V, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(V, K0 + V, dtype=torch.bfloat16, device=DEV)
    x[:, :K0] = torch.rand(T, K0, generator=g, device=DEV).bfloat16()
    w[:, :K0] = (torch.rand(V, K0, generator=g, device=DEV) * 120 / K0).bfloat16()
    z = torch.stack([x.double() @ v.double() for v in w], 1)            # 30 each, all terms positive
    w[:, K0:] = torch.eye(V, device=DEV).bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device=DEV)
    lse = torch.logsumexp(z, 1).float()
    d = torch.rand(T, generator=g, device=DEV) + 0.5
    dx, _ = wpg.lora_ce_bwd(x, w, y, lse, d, need_dW=False, dX_dtype=torch.float32)
    G = torch.exp(z - lse.double()[:, None]) * d.double()[:, None]
    others = torch.arange(V, device=DEV)[None, :] != y[:, None]
    # an entry beside the target's: one rounding to bf16, the logit's error, and what check_bwd counts for the
    # exponential; the row's own factor is in it twice, once over itself
    rel = U16 * (1 + U16) + 1.01 * (units(K0) * z + 2.0 ** -18)
    off = ((dx[:, K0:].double() - G).abs() / (rel * G))[others]
    assert float(off.max()) <= 1


def test_weight_gradient_of_many_rows():
    # z = 0 against two entries: G over its row's factor is -1 and 1, the factor times X exact in bf16
    T, K = 1 << 20, 64
    g = torch.Generator(device=DEV).manual_seed(3)
    x = (torch.rand(T, K, generator=g, device=DEV) + 0.5).bfloat16()
    w = torch.zeros(2, K, dtype=torch.bfloat16, device=DEV)
    y = torch.zeros(T, dtype=torch.int64, device=DEV)
    lse = torch.full((T,), float(np.log(2)), device=DEV)
    d = torch.ones(T, device=DEV)
    _, dw = wpg.lora_ce_bwd(x, w, y, lse, d, need_dX=False, dW_dtype=torch.float32)
    want = 0.5 * x.double().sum(0)
    # 2^-22: 1 - p from the fp32 lse, which may be off by half a step
    off = torch.stack([-dw[0], dw[1]]).double() / want - 1
    assert float(off.abs().max()) <= units(T) + 2.0 ** -22, float(off.abs().max())


def test_row_gradient_of_many_entries():
    # X = 0: every entry but the target's has p over 1 - p = 2^-18, exact in bf16; columns enough that the contraction is
    # not split
    T, K, V = 64, 19456, (1 << 18) + 1
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    w = torch.empty(V, K, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    total = torch.zeros(K, dtype=torch.float64, device=DEV)
    for a in range(0, V, 16384):
        part = (torch.rand(min(16384, V - a), K, generator=g, device=DEV) + 0.5).bfloat16()
        w[a:a + len(part)] = part
        total += part.double().sum(0)
    y = torch.arange(T, device=DEV) * 4001
    lse = torch.full((T,), float(np.log(V)), device=DEV)
    dx, _ = wpg.lora_ce_bwd(x, w, y, lse, torch.ones(T, device=DEV), need_dW=False, dX_dtype=torch.float32)
    mean, own = (total - w[y].double()) / (V - 1), w[y].double()
    want = (mean - own) * (1 - 1 / V)
    # the target's entry is one term of the sum; p from the fp32 lse (half a step of 12.5: 2^-21 and the exponential's
    # 2^-22) moves each factor
    bound = (units(V) + 2.0 ** -19) * (mean + own)
    assert bool(((dx.double() - want).abs() <= bound).all()), float(((dx.double() - want).abs() / bound).max())
