"""The adapter-set kernels over enough work that every CTA takes its loop several times: rings that wrap,
accumulators used in turn, sums carried from turn to turn, and a last turn that is not whole.  Sizes
follow the device's SM count."""
import numpy as np
import pytest
import torch

import weight_patches_gb300 as wpg
from tests import gpu_util as gu
from tests import test_gpu_adamw as ta
from tests import test_gpu_multi as tm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------------------------ norms
# The definition in float64 on the device and the bounds of test_gpu_norm.py; only the column sums' chains are
# counted anew: a CTA (at least one per SM) adds its rows in turn, the second kernel adds at most 16 CTAs per
# SM in 64 threads, and those 64: T / SMs + 4 + 16 SMs / 64 + 64 additions.

def _rows(C, size):
    """Rows with which each CTA fills its ring (at most 220 KiB and 8 stages of 4 rows and 16 CTAs per SM) and
    then takes two turns more of at most 4 rows (at most 16 warps per SM, a warp at most 8 vectors a lane)."""
    warps = -(-C * size // (16 * 8 * 32))
    ring = min(8 * 4 * 16, 220 * 1024 // (C * size))
    return _sms() * (ring + 2 * 4 * max(1, 16 // warps)) + 3


def _ulp(dtype, v):
    """Spacing of dtype's values around v."""
    bits = 8 if dtype == torch.bfloat16 else 24
    _, e = torch.frexp(v.abs().clamp(min=2.0 ** -126))
    return torch.ldexp(torch.ones_like(v), e - bits)


def _assert_within(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    if bool(bad.any()):
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first {i}: {float(got[i])}, "
                             f"want {float(want[i])} within {float(bound[i])}")


def _norm_case(T, C, dtype, kind, ld, off, seed=0):
    g = torch.Generator(device=gu.DEV).manual_seed(seed)
    layer = kind == wpg.WP_NORM_LAYER

    def rows(shift):
        buf = torch.full((off + T * ld + 16,), float("nan"), dtype=dtype, device=gu.DEV)
        x = buf[off:off + T * ld].view(T, ld)[:, :C]
        x.copy_(torch.randn(T, C, generator=g, device=gu.DEV) * (0.5 + torch.rand(T, 1, generator=g, device=gu.DEV)) + shift)
        return x

    x, dy = rows(0.3), rows(0.0)
    w = (1 + 0.2 * torch.randn(C, generator=g, device=gu.DEV)).to(dtype)
    b = 0.2 * torch.randn(C, generator=g, device=gu.DEV)
    eps = 1e-5
    out = torch.full((off + T * ld + 16,), 7.0, dtype=dtype, device=gu.DEV)
    y, stats = wpg.lora_norm_fwd(x, w, b, eps, kind, out=out[off:off + T * ld].view(T, ld)[:, :C])
    dx, dw, db = wpg.lora_norm_bwd(dy, x, w, stats, kind)
    torch.cuda.synchronize()
    assert wpg.lora_device_status() == 0

    # forward
    gam = (64 + 5 + 16 + C / 512 + 4) * U
    X, W = x.double(), w.double()
    mu = X.mean(1, keepdim=True) if layer else torch.zeros(T, 1, dtype=torch.float64, device=gu.DEV)
    d = X - mu
    var, dist = (d * d).mean(1, keepdim=True), d.abs().mean(1, keepdim=True)
    r = (var + eps).rsqrt()
    emu = gam * X.abs().mean(1, keepdim=True) if layer else torch.zeros_like(mu)
    rel_r = 0.5 * ((var * (gam + 4 * U) + emu ** 2 + 2 * emu * dist * gam + 2 * U * emu * dist) / (var + eps) + 2 * U) + 4 * U
    _assert_within(stats[0], mu[:, 0], (emu + _ulp(torch.float32, mu))[:, 0], "mean")
    _assert_within(stats[1], r[:, 0], (rel_r * r + _ulp(torch.float32, r))[:, 0], "rstd")
    want = d * r * W + b.double()
    e = (d * r * W).abs() * (rel_r + 4 * U) + r * W.abs() * emu + 2 * U * want.abs() + 2 * U * b.double().abs()
    _assert_within(y, want, _ulp(dtype, want.abs() + e) + e, "y")
    del want, e, d
    y.fill_(7.0)
    assert bool((out == 7.0).all())
    # backward, from the statistics as they were saved
    mu, r = stats[0].double()[:, None], stats[1].double()[:, None]
    xh, D = (X - mu) * r, dy.double()
    h = D * W
    m1 = h.mean(1, keepdim=True) if layer else 0.0
    want = r * (h - m1 - xh * (h * xh).mean(1, keepdim=True))
    a1 = h.abs().mean(1, keepdim=True) if layer else 0.0
    a2 = (h * xh).abs().mean(1, keepdim=True)
    e = r * ((gam + 8 * U) * (a1 + xh.abs() * a2) + 6 * U * (h.abs() + xh.abs() * a2))
    _assert_within(dx, want, _ulp(dtype, want.abs() + e) + e, "dx")
    chain = (T / _sms() + 4 + 16 * _sms() / 64 + 64) * U
    for got, terms, what in ((dw, D * xh, "dw"), (db, D, "db")):
        want, e = terms.sum(0), (chain + 3 * U) * terms.abs().sum(0)
        _assert_within(got, want, _ulp(torch.float32, want.abs() + e) + e, what)
    again = wpg.lora_norm_bwd(dy, x, w, stats, kind)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [24, 200, 256, 512, 1536, 2048, 2560, 4096, 6144, 8192, 12288, 14336, 16384, 20480])
def test_aligned_rows(C, dtype):
    T = _rows(C, 2 if dtype == torch.bfloat16 else 4)
    _norm_case(T, C, dtype, wpg.WP_NORM_LAYER, C, 0)
    _norm_case(T, C, dtype, wpg.WP_NORM_RMS, C + 16, 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C", [1, 7, 31, 255, 509, 1025, 2187, 4099, 6001, 8191, 12001, 16001])
def test_shifted_rows(C, dtype):
    T = _rows(C, 2 if dtype == torch.bfloat16 else 4)
    _norm_case(T, C, dtype, wpg.WP_NORM_LAYER, C, 3)
    _norm_case(T, C, dtype, wpg.WP_NORM_RMS, C + 5, 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", [wpg.WP_NORM_LAYER, wpg.WP_NORM_RMS])
def test_long_rows(kind, dtype):
    _norm_case(4 * _sms() + 5, 33001, dtype, kind, 33002, 1)       # four CTAs per SM, two in the backward


# ------------------------------------------------------------------------------ many adapters
@pytest.mark.parametrize("base,T", [("bf16", 1500), ("nf4", 2700), (None, 1500)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_many_rows_and_columns(base, T, out):
    # blocks without an adapter, of one slot, in runs, and in any order, side by side
    lay = tm.Layer(T, 512, 9000, 1, 40, 12, base=base, bias="bf16", seed=T)
    slot = tm._slots(T, 12, "any", 1)
    slot[256:512] = [-1] * 256
    slot[512:700] = [3] * 188
    slot[700:1100] = tm._slots(400, 12, "runs", 2)
    y = lay.check(slot, 0.8, out_dtype=out)
    assert torch.equal(lay.run(slot, 0.8, out_dtype=out), y)


@pytest.mark.parametrize("T", [1, 16, 40, 64, 100, 128])
def test_a_wide_4_bit_weight(T):
    lay = tm.Layer(T, 1024, 28672, 2, 16, 6, base="nf4", seed=T)
    slot = tm._slots(T, 6, "any", T)
    y = lay.check(slot)
    assert torch.equal(lay.run(slot), y)


# ------------------------------------------------------------------------------ AdamW
@pytest.mark.parametrize("param", ["fp32", "bf16", "master"])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
def test_moments_of_both_kinds_in_one_large_set(param, grad):
    # more units of 2048 elements than CTAs run at a time (four per SM), ragged ends, missing gradients
    n = 2 * _sms() * 2048
    a = ta.Set([n + 77, 3, 2048 * 20, n - 1000, 0, n + 2047, 511], param, 8, grad, seed=1)
    b = ta.Set([5000, n // 2 + 1, 2048, 1, 70001, 9, 12], param, 32, grad, seed=2)
    order = [s for pair in zip(((a, i) for i in range(7)), ((b, i) for i in range(7))) for s in pair]
    lists = {id(s): (s.cut(s.p), s.ml, s.vl, s.cut(s.master) or [None] * 7, s.cut(s.g)) for s in (a, b)}
    p, m, v, ma, g = ([lists[id(s)][k][i] for s, i in order] for k in range(5))
    plan = wpg.lora_adamw_plan(p, m, v, masters=ma)
    g[order.index((a, 2))] = g[order.index((b, 4))] = None
    for t in (1, 2, 50):
        before = a.snapshot(), b.snapshot()
        wpg.lora_adamw_step(plan, g, step=t, **ta.HYPER)
        ta._check(a, before[0], t, skip=(2,))
        ta._check(b, before[1], t, skip=(4,))


def test_many_8_bit_tensors_cross_the_launches():
    s = ta.Set([3 + i % 300 for i in range(4000)], "master", 8, gap=0)
    for t in (1, 2):
        before = s.snapshot()
        grads = s.cut(s.g)
        grads[7] = grads[3899] = grads[3900] = None
        wpg.lora_adamw_step(s.plan, grads, step=t, **ta.HYPER)
        ta._check(s, before, t, skip=(7, 3899, 3900))


def test_decode_of_many_blocks():
    n = 8192 * 8 * _sms() + 1001                     # 8192 codes a CTA
    q = torch.randint(0, 256, (n,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(torch.uint8)
    top = torch.rand((n + 255) // 256, generator=torch.Generator().manual_seed(4)) * 3
    got = wpg.lora_block8_decode(q.to(gu.DEV), top.to(gu.DEV)).cpu().numpy()
    assert np.array_equal(got, ta.oa.decode(q.numpy(), top.numpy(), False))
