"""lora_ce_fwd with rows of several chunks of columns (more than 1024 of more than 256 rows) against the 64-bit definition."""
import numpy as np
import pytest
import torch

import weight_patches_gb300 as wpg
from oracle import ce as oce
from tests.test_gpu_ce import DEV, U32, case, check_fwd, f64

pytestmark = pytest.mark.gpu


# A logit's error, as test_gpu_ce.logit_error has it but for the chunks' number: 1024 products each.
def units(n):
    return (2.125 * min(n, 1024) + n / 1024 + 4) * U32


@pytest.mark.parametrize("T,K,V", [(300, 1032, 700), (300, 2056, 513), (257, 4096, 1000), (512, 1024, 300), (270, 5120, 257)])
def test_forward(T, K, V):
    check_fwd(*case(T, K, V, seed=T + K, ignored=0.1))


def test_forward_units_of_several_tiles_of_several_chunks():
    # 8 row blocks of 305 tiles each over 76 pairs: units of two tiles, each of two chunks
    x, w, y = case(2048, 1160, 78000, seed=3, ignored=0.1)
    loss, lse = wpg.lora_ce_fwd(x, w, y)
    keep = (y >= 0) & (y < len(w))
    wd = w.double()
    for a in range(0, 2048, 512):
        xd, at = x[a:a + 512].double(), y[a:a + 512].clamp(0, len(w) - 1)
        z = xd @ wd.t()
        want = torch.logsumexp(z, 1)
        # as in check_fwd: twice a logit's error, the sum of exponentials, and roundings of lse's own size
        e = units(1160) * (xd.abs() @ wd.abs().t()).amax(1)
        bound = 2 * e + (16 + 64 + len(w) / 128) * U32 + 8 * U32 * (want.abs() + 1)
        k = keep[a:a + 512]
        assert bool(((lse[a:a + 512] - want).abs() <= bound)[k].all())
        assert bool(((loss[a:a + 512] - (want - z.gather(1, at[:, None])[:, 0])).abs() <= 2 * bound)[k].all())
    assert bool((loss[~keep] == 0).all())


def test_loss_of_wide_rows_past_32_bits():
    # rows of more than 2^31 elements in all: the last ones' loss against that of a call of their own
    T, K, V = 270_001, 8192, 40
    xs, w, ys = case(70, K, V, seed=30)
    x = torch.zeros(T, K, dtype=torch.bfloat16, device=DEV)
    x[-70:] = xs
    y = torch.full((T,), -100, device=DEV)
    y[-70:], y[:600] = ys, 1
    loss, lse = wpg.lora_ce_fwd(x, w, y)
    want, wlse = oce.forward(f64(xs), f64(w), ys.cpu().numpy())
    e = units(K) * (np.abs(f64(xs)) @ np.abs(f64(w)).T).max(axis=1)
    bound = 2 * e + 80 * U32 + 8 * U32 * (np.abs(wlse) + 1)
    assert np.all(np.abs(f64(lse[-70:]) - wlse) <= bound) and np.all(np.abs(f64(loss[-70:]) - want) <= 2 * bound)


# all terms positive and alike, so that cuts add up in one direction
@pytest.mark.parametrize("T", [8, 300])
def test_forward_of_very_long_rows(T):
    K, V = 1 << 20, 40
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.rand(T, K, generator=g, device=DEV).bfloat16()
    w = (torch.rand(V, K, generator=g, device=DEV) * 120 / K).bfloat16()
    y = torch.randint(0, V, (T,), generator=g, device=DEV)
    loss, lse = wpg.lora_ce_fwd(x, w, y)
    z = torch.stack([x.double() @ v.double() for v in w], 1)
    want = torch.logsumexp(z, 1)
    # (a few rows' chunks are 64 to 256 products: more of them, each cut less)
    e = (units(K) + K / 64 * U32 * (T <= 256)) * z.amax(1)
    bound = 2 * e + 80 * U32 + 8 * U32 * (want.abs() + 1)
    assert bool(((lse - want).abs() <= bound).all())
    assert bool(((loss - (want - z.gather(1, y[:, None])[:, 0])).abs() <= 2 * bound).all())
