"""Norm forward and backward against the FP64 definition, element by element.

u = 2^-24.  A row sum of n terms is taken by at least 32 threads, each adding its terms in turn
(at most 64 in registers, n / 512 in the long form), then 5 shuffles and at most 16 warps:
gamma = (64 + 5 + 16 + n / 512 + 4) u of the sum of magnitudes covers it.
  mu:  |err| <= gamma mean|x|
  r:   the variance's relative error is gamma + 4u, plus the squared error of mu (and twice its
       product with the mean distance, which is zero for the exact mu up to gamma): r's is half of
       that plus 4u for root, quotient and eps
  y:   |y| err <= |xh w| (rel(r) + 4u) + r |w| err(mu) + 2u |y|, then one output rounding
  dx:  xh carries 2u; m1, m2 carry (gamma + 6u) of their sums of magnitudes
  dw, db: sums over T rows, (T + 64) u of the sum of magnitudes plus 3u for the terms
"""
import numpy as np
import pytest
import torch

import weight_patches_gb300 as wpg
from oracle import norm as on
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
KINDS = [wpg.WP_NORM_LAYER, wpg.WP_NORM_RMS]


def _data(T, C, dtype, seed, shift=0.3, ld=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, C, generator=g) * (0.5 + torch.rand(T, 1, generator=g)) + shift
    full = torch.full((T, ld or C), float("nan"), dtype=dtype)
    full[:, :C] = x.to(dtype)
    return full.to(gu.DEV)[:, :C]


def _vec(C, dtype, seed, base):
    g = torch.Generator().manual_seed(seed)
    return (base + 0.2 * torch.randn(C, generator=g)).to(dtype).to(gu.DEV)


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _ulp(dtype, v):
    return gu.ulp_bf16(v) if dtype == torch.bfloat16 else gu.ulp_f32(v)


def _gamma(C):
    return (64 + 5 + 16 + C / 512 + 4) * U


def _check_fwd(x, w, b, kind, eps, y, stats):
    layer = kind == wpg.WP_NORM_LAYER
    X, wf, bf = _f64(x), _f64(w), _f64(b)
    C = X.shape[1]
    want, mu, r = on.forward(X, wf, bf, eps, layer)
    gam = _gamma(C)
    emu = gam * np.abs(X).mean(1) if layer else np.zeros(X.shape[0])
    var = ((X - mu[:, None]) ** 2).mean(1)
    dist = np.abs(X - mu[:, None]).mean(1)
    rel_var = (var * (gam + 4 * U) + emu ** 2 + 2 * emu * dist * gam + 2 * U * emu * dist) / (var + eps) + 2 * U
    rel_r = 0.5 * rel_var + 4 * U
    st = _f64(stats)
    gu.assert_elementwise(st[0], mu, emu + gu.ulp_f32(mu), "mean")
    gu.assert_elementwise(st[1], r, rel_r * r + gu.ulp_f32(r), "rstd")
    aw = np.ones(C) if wf is None else np.abs(wf)
    xh = np.abs(X - mu[:, None]) * r[:, None]
    e = xh * aw * (rel_r[:, None] + 4 * U) + r[:, None] * aw * emu[:, None] + 2 * U * np.abs(want) \
        + (0 if bf is None else 2 * U * np.abs(bf))
    gu.assert_elementwise(_f64(y), want, _ulp(y.dtype, np.abs(want) + e) + e, "y")


# lengths of one, below and across the register forms' capacities (256, 512, 1024, 4096, 8192,
# 16384, 32768 elements), odd ones, and beyond them
SHAPES = [(1, 1), (3, 7), (5, 64), (2, 255), (9, 256), (4, 513), (7, 1024), (33, 1536), (8, 1537), (3, 2048),
          (3, 2056), (5, 4099), (2, 5120), (2, 8192), (2, 8200), (3, 14336), (1, 16385), (2, 32768), (2, 32776),
          (1, 40001), (700, 24)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,C", SHAPES)
def test_forward(T, C, dtype, kind):
    x = _data(T, C, dtype, 1)
    w, b = _vec(C, dtype, 2, 1.0), _vec(C, torch.float32, 3, 0.0)
    y, stats = wpg.lora_norm_fwd(x, w, b, 1e-5, kind)
    _check_fwd(x, w, b, kind, 1e-5, y, stats)
    y, stats = wpg.lora_norm_fwd(x, None, None, 1e-5, kind)
    _check_fwd(x, None, None, kind, 1e-5, y, stats)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C,ld,off", [(1536, 1544, 0), (1536, 1540, 0), (96, 104, 3), (33, 50, 1), (4099, 4104, 5)])
def test_strides_and_offsets_and_canaries(C, ld, off, dtype):
    T = 6
    x = _data(T, C + off, dtype, 4, ld=ld + off)[:, off:]
    out = torch.full((T + 2, ld + 9), 7.0, dtype=dtype, device=gu.DEV)
    y, stats = wpg.lora_norm_fwd(x, None, None, 1e-5, out=out[1:T + 1, 1:C + 1])
    _check_fwd(x, None, None, wpg.WP_NORM_LAYER, 1e-5, y, stats)
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1:T + 1, 1:C + 1] = False
    assert bool((out[keep] == 7.0).all())
    dy = _data(T, C, dtype, 5, shift=0.0)
    _check_bwd(dy, x, None, wpg.WP_NORM_LAYER, stats)


def test_large_mean_keeps_its_digits():
    x = _data(4, 3000, torch.float32, 6, shift=1000.0)
    y, stats = wpg.lora_norm_fwd(x, None, None, 1e-6)
    _check_fwd(x, None, None, wpg.WP_NORM_LAYER, 1e-6, y, stats)


def test_constant_and_zero_rows():
    x = torch.zeros(3, 128, device=gu.DEV)
    x[1] = 5.0
    w, b = _vec(128, torch.float32, 2, 1.0), _vec(128, torch.float32, 3, 0.0)
    y, stats = wpg.lora_norm_fwd(x, w, b, 1e-5)
    assert torch.equal(y, b.expand(3, 128))
    assert torch.equal(stats[0], torch.tensor([0.0, 5.0, 0.0], device=gu.DEV))


def test_a_row_that_is_not_finite_stays_its_own():
    x = _data(16, 512, torch.bfloat16, 8)
    clean, _ = wpg.lora_norm_fwd(x)
    bad = x.clone()
    bad[3, 17] = float("inf")
    bad[9, 0] = float("nan")
    y, _ = wpg.lora_norm_fwd(bad)
    rows = [i for i in range(16) if i not in (3, 9)]
    assert torch.equal(y[rows], clean[rows])
    assert bool(y[3].isnan().any()) and bool(y[9].isnan().all())


def _check_bwd(dy, x, w, kind, stats, ws=None):
    layer = kind == wpg.WP_NORM_LAYER
    dx, dw, db = wpg.lora_norm_bwd(dy, x, w, stats, kind, workspace=ws)
    X, D, wf, st = _f64(x), _f64(dy), _f64(w), _f64(stats)
    mu = st[0] if layer else np.zeros(X.shape[0])
    T, C = X.shape
    gdx, gdw, gdb = on.backward(D, X, wf, mu, st[1], layer)
    gam = _gamma(C)
    xh = np.abs(X - mu[:, None]) * st[1][:, None]
    h = np.abs(D) if wf is None else np.abs(D * wf)
    m1 = h.mean(1, keepdims=True) if layer else 0.0
    m2 = (h * xh).mean(1, keepdims=True)
    e = st[1][:, None] * ((gam + 8 * U) * (m1 + xh * m2) + 6 * U * (h + xh * m2))
    gu.assert_elementwise(_f64(dx), gdx, _ulp(dx.dtype, np.abs(gdx) + e) + e, "dx")
    ew = ((T + 64) * U + 3 * U) * (np.abs(D) * xh).sum(0)
    eb = (T + 64) * U * np.abs(D).sum(0)
    gu.assert_elementwise(_f64(dw), gdw, gu.ulp_f32(np.abs(gdw) + ew) + ew, "dw")
    gu.assert_elementwise(_f64(db), gdb, gu.ulp_f32(np.abs(gdb) + eb) + eb, "db")
    return dx, dw, db


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,C", SHAPES + [(2000, 136), (1300, 40)])
def test_backward(T, C, dtype, kind):
    x, dy = _data(T, C, dtype, 11), _data(T, C, dtype, 12, shift=0.1)
    w = _vec(C, dtype, 13, 1.0)
    _, stats = wpg.lora_norm_fwd(x, w, None, 1e-5, kind)
    dx, dw, db = _check_bwd(dy, x, w, kind, stats)
    # the same bits again, and each output alone
    again = wpg.lora_norm_bwd(dy, x, w, stats, kind)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))
    only, none, none2 = wpg.lora_norm_bwd(dy, x, w, stats, kind, need_dw=False, need_db=False)
    assert torch.equal(only, dx) and none is None and none2 is None
    _, dw2, _ = wpg.lora_norm_bwd(dy, x, w, stats, kind, need_dx=False, need_db=False)
    assert torch.equal(dw2, dw)


@pytest.mark.parametrize("kind", KINDS)
def test_backward_against_differences(kind):
    T, C, eps, step = 3, 24, 1e-5, 1e-6
    layer = kind == wpg.WP_NORM_LAYER
    x, dy, w = _data(T, C, torch.float32, 21), _data(T, C, torch.float32, 22, 0.0), _vec(C, torch.float32, 23, 1.0)
    _, stats = wpg.lora_norm_fwd(x, w, None, eps, kind)
    dx, dw, db = wpg.lora_norm_bwd(dy, x, w, stats, kind)
    X, D, W = _f64(x), _f64(dy), _f64(w)
    loss = lambda X, W, b: float((on.forward(X, W, b, eps, layer)[0] * D).sum())  # noqa: E731
    zero = np.zeros(C)
    for got, at in ((dx, "x"), (dw, "w"), (db, "b")):
        base = {"x": X, "w": W, "b": zero}
        num = np.zeros_like(base[at])
        for i in np.ndindex(*num.shape):
            v = []
            for s in (step, -step):
                q = {k: a.copy() for k, a in base.items()}
                q[at][i] += s
                v.append(loss(q["x"], q["w"], q["b"]))
            num[i] = (v[0] - v[1]) / (2 * step)
        # the difference's own error: step^2 of the third derivative and the rounding 2^-52 |loss| /
        # step, both below 1e-8; the kernel's fp32 result carries some 1e-6 of its terms (below 10)
        assert np.abs(_f64(got) - num).max() < 1e-4


def test_no_rows_and_other_stream():
    x = torch.empty(0, 64, device=gu.DEV)
    y, stats = wpg.lora_norm_fwd(x)
    assert y.shape == (0, 64)
    dx, dw, db = wpg.lora_norm_bwd(x, x, None, stats)
    assert dx.shape == (0, 64) and float(dw.abs().sum() + db.abs().sum()) == 0.0
    x = _data(300, 777, torch.bfloat16, 31)
    want, st0 = wpg.lora_norm_fwd(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got, st1 = wpg.lora_norm_fwd(x)
        grads = wpg.lora_norm_bwd(x, x, None, st1)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want) and torch.equal(st0, st1)
    assert all(torch.equal(a, b) for a, b in zip(grads, wpg.lora_norm_bwd(x, x, None, st0)))


def _placed(T, C, ld, off, dtype, seed, shift=0.3):
    """[T, C] rows ld apart, the first `off` elements past a 256-byte boundary, NaN around them."""
    buf = torch.full((off + T * ld + 64,), float("nan"), dtype=dtype, device=gu.DEV)
    x = buf[off:off + T * ld].view(T, ld)[:, :C]
    x.copy_(_data(T, C, dtype, seed, shift))
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,C", [(T, C) for T in (1, 2, 3, 4, 5, 9)
                                 for C in (1, 2, 3, 5, 8, 9, 31, 63, 255, 263, 511, 1025, 2051, 4095, 8191, 16001)]
                         + [(1300, C) for C in (1, 3, 8, 31, 255)])
def test_rows_at_any_place(T, C, dtype):
    for i, gap in enumerate((0, 0, 5)):              # rows one after another, and apart
        x = _placed(T, C, C + gap, (0, 3, 6)[i], dtype, 1)
        dy = _placed(T, C, C + (gap + 3 if gap else 0), (5, 0, 1)[i], dtype, 2, 0.0)
        w, b = _vec(C + 1, dtype, 3, 1.0)[i % 2:][:C], _vec(C + 2, torch.float32, 4, 0.0)[i:][:C]
        off, ld = (7, 2, 4)[i], C + (gap and 11)
        out = torch.full((off + T * ld + 64,), 7.0, dtype=dtype, device=gu.DEV)
        y, stats = wpg.lora_norm_fwd(x, w, b, 1e-5, out=out[off:off + T * ld].view(T, ld)[:, :C])
        _check_fwd(x, w, b, wpg.WP_NORM_LAYER, 1e-5, y, stats)
        y.fill_(7.0)
        assert bool((out == 7.0).all())
        _check_bwd(dy, x, w, wpg.WP_NORM_LAYER, stats)
