"""The adapter-set operators refuse bad arguments on the host (nothing is launched: no GPU needed),
and the binding refuses tensors of the wrong kind."""
import ctypes
import math

import numpy as np
import pytest
import torch

import weight_patches_gb300 as wpg
from oracle import adamw as oa
from oracle import norm as on

FAKE = 0x10000
BF, F32, NF4 = wpg.WP_BF16, wpg.WP_FP32, wpg.WP_NF4


@pytest.fixture(scope="module")
def lib():
    return wpg.lib()


def _m(rows, cols, dtype=BF, ld=None, data=FAKE, absmax=None):
    return wpg.WpMat(data, dtype, rows, cols, cols if ld is None else ld, absmax)


def _o(rows, cols, dtype=BF, ld=None, data=FAKE):
    return wpg.WpOut(data, dtype, rows, cols, cols if ld is None else ld)


def _bank(S=4, G=1, R=16, K=128, N=256, dtype=BF, A=FAKE, B=FAKE, scale=FAKE):
    return wpg.WpBank(A, B, scale, dtype, S, G, R, K, N)


def _r(x):
    return None if x is None else ctypes.byref(x)


def _multi(lib, X=None, W="w", bias=None, bank=None, slot=FAKE, rows=None, rs=1.0, Y=None, ws=FAKE, nbytes=1 << 40):
    W = _m(256, 128) if isinstance(W, str) else W
    return lib.lora_linear_fwd_multi(_r(X or _m(9, 128)), _r(W), _r(bias), _r(bank or _bank()), slot, rows, rs,
                                     _r(Y or _o(9, 256)), ws, nbytes, None)


def test_multi_refusals(lib):
    assert _multi(lib, X=_m(9, 128, F32)) == -3
    assert _multi(lib, bank=_bank(dtype=F32)) == -3
    assert _multi(lib, W=_m(256, 128, F32)) == -3
    assert _multi(lib, bank=_bank(K=136)) == -2                     # bank's inner size
    assert _multi(lib, bank=_bank(N=264)) == -2                     # W rows
    assert _multi(lib, bank=_bank(G=3)) == -2                       # 256 % 3
    assert _multi(lib, bank=_bank(R=12)) == -2                      # rank % 8
    assert _multi(lib, bank=_bank(R=264)) == -8
    assert _multi(lib, bank=_bank(G=16)) == -8
    assert _multi(lib, bank=_bank(S=0)) == -1
    assert _multi(lib, bank=_bank(A=None)) == -1
    assert _multi(lib, bank=_bank(scale=None)) == -1
    assert _multi(lib, bank=_bank(B=FAKE + 2)) == -4
    assert _multi(lib, slot=None) == -1
    assert _multi(lib, rs=math.nan) == -1 and _multi(lib, rs=math.inf) == -1 and _multi(lib, rs=1e300) == -1
    assert _multi(lib, Y=_o(9, 255)) == -2 and _multi(lib, Y=_o(8, 256)) == -2
    assert _multi(lib, Y=_o(9, 256, NF4)) == -1
    assert _multi(lib, Y=_o(9, 256, ld=260)) == -4
    assert _multi(lib, X=_m(9, 128, ld=132)) == -4
    assert _multi(lib, X=_m(9, 128, data=FAKE + 8)) == -4
    assert _multi(lib, X=_m(9, 124), bank=_bank(K=124), W=_m(256, 124)) == -4
    assert _multi(lib, W=_m(256, 128, ld=130)) == -4
    assert _multi(lib, W=_m(256, 128, NF4)) == -1                   # no block scales
    assert _multi(lib, bias=_m(1, 255)) == -2 and _multi(lib, bias=_m(1, 256, data=None)) == -1
    assert _multi(lib, ws=None) == -5 and _multi(lib, nbytes=16) == -5
    assert _multi(lib, ws=FAKE + 4) == -4
    assert lib.lora_linear_fwd_multi(None, None, None, None, None, None, 1.0, None, None, 0, None) == -1
    # no rows: nothing to do, null pointers are fine
    assert _multi(lib, X=_m(0, 128, data=None), Y=_o(0, 256, data=None), slot=None, ws=None, nbytes=0) == 0


def test_multi_workspace_size(lib):
    f = lambda X, W, b: lib.lora_multi_workspace_size(_r(X), _r(W), _r(b))  # noqa: E731
    assert f(_m(9, 128), _m(256, 128), _bank()) > 0
    assert f(_m(0, 128, data=None), _m(256, 128), _bank()) == 0
    assert f(_m(9, 128), _m(256, 120), _bank()) == 0
    assert f(None, None, None) == 0


def test_norm_refusals(lib):
    fwd = lambda X=_m(5, 64), w=None, b=None, kind=0, eps=1e-5, Y=_o(5, 64): lib.lora_norm_fwd(  # noqa: E731
        _r(X), _r(w), _r(b), kind, eps, _r(Y), None, None)
    assert fwd(kind=2) == -1 and fwd(eps=-1.0) == -1 and fwd(eps=math.nan) == -1
    assert fwd(X=None) == -1 and fwd(Y=None) == -1
    assert fwd(X=_m(5, 64, NF4)) == -1
    assert fwd(Y=_o(5, 64, F32)) == -3
    assert fwd(Y=_o(5, 63)) == -2 and fwd(Y=_o(4, 64)) == -2
    assert fwd(X=_m(5, 64, ld=60)) == -1
    assert fwd(w=_m(1, 63)) == -2 and fwd(w=_m(1, 64, data=None)) == -1 and fwd(b=_m(1, 65)) == -2
    assert fwd(X=_m(0, 64, data=None), Y=_o(0, 64, data=None)) == 0

    def bwd(dY=_m(5, 64), X=_m(5, 64), w=None, stats=FAKE, kind=0, dX=_o(5, 64), dW=_o(1, 64, F32), dB=None, ws=FAKE,
            nbytes=1 << 30):
        return lib.lora_norm_bwd(_r(dY), _r(X), _r(w), stats, kind, _r(dX), _r(dW), _r(dB), ws, nbytes, None)
    assert bwd(stats=None) == -1 and bwd(kind=-1) == -1
    assert bwd(dY=_m(5, 64, F32)) == -3 and bwd(dX=_o(5, 64, F32)) == -3 and bwd(dW=_o(1, 64)) == -3
    assert bwd(dY=_m(5, 65)) == -2 and bwd(dX=_o(6, 64)) == -2 and bwd(dW=_o(1, 65, F32)) == -2
    assert bwd(dB=_o(1, 64, F32, data=None)) == -1
    assert bwd(ws=None) == -5 and bwd(nbytes=8) == -5 and bwd(ws=FAKE + 4) == -4
    assert bwd(dX=None, dW=None) == 0
    need = lib.lora_workspace_size(wpg.WP_OP_NORM_BWD, _r(_m(5, 64)), None, None, 0)
    assert need >= 2 * 64 * 4


def _t(numel=100, dtype=F32, bits=32, **kw):
    base = dict(param=FAKE, master=None, m=FAKE, v=FAKE, m_absmax=FAKE, v_absmax=FAKE)
    base.update(kw)
    return wpg.WpAdamWTensor(base["param"], base["master"], base["m"], base["v"], base["m_absmax"], base["v_absmax"],
                             numel, dtype, bits)


def test_adamw_refusals(lib):
    def init(t, n=1, table=FAKE, nbytes=1 << 20):
        arr = (wpg.WpAdamWTensor * 1)(t)
        return lib.lora_adamw_plan_init(arr, n, table, nbytes, ctypes.byref(wpg.WpAdamWPlan()), None)
    assert init(_t(-1)) == -1 and init(_t(param=None)) == -1 and init(_t(m=None)) == -1
    assert init(_t(bits=8, v_absmax=None)) == -1
    assert init(_t(dtype=NF4)) == -3 and init(_t(bits=16)) == -3 and init(_t(master=FAKE)) == -3
    assert init(_t(param=FAKE + 2)) == -4 and init(_t(m=FAKE + 1)) == -4
    assert init(_t(), n=0) == -1 and init(_t(), n=62401) == -8
    assert init(_t(), table=None) == -5 and init(_t(), nbytes=100) == -5 and init(_t(), table=FAKE + 8) == -4
    arr = (wpg.WpAdamWTensor * 1)(_t(param=None))
    assert lib.lora_adamw_plan_size(arr, 1) == 0 and lib.lora_adamw_plan_size(None, 1) == 0

    plan = wpg.WpAdamWPlan(FAKE, 1, 1, (ctypes.c_int64 * 17)())
    grads = (ctypes.c_void_p * 1)(None)

    def step(dtype=F32, g=grads, p=plan, **kw):
        a = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, wd=0.0, gs=1.0, step=1)
        a.update(kw)
        args = wpg.WpAdamWArgs(a["lr"], a["beta1"], a["beta2"], a["eps"], a["wd"], a["gs"], a["step"], None)
        return lib.lora_adamw_step(_r(p), g, dtype, ctypes.byref(args), None)
    assert step(dtype=NF4) == -3
    for bad in (dict(lr=math.nan), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(eps=-1e-9),
                dict(wd=math.inf), dict(gs=math.nan), dict(step=0)):
        assert step(**bad) == -1, bad
    assert step(g=(ctypes.c_void_p * 1)(FAKE + 2)) == -4
    assert step(p=wpg.WpAdamWPlan(None, 1, 1, (ctypes.c_int64 * 17)())) == -1
    assert step(p=wpg.WpAdamWPlan(FAKE, 1, 2, (ctypes.c_int64 * 17)())) == -1
    assert step() == 0                                               # an empty unit range: nothing to launch
    assert lib.lora_block8_decode(None, 1, FAKE, 5, FAKE, None) == -1
    assert lib.lora_block8_decode(FAKE, 1, FAKE, -1, FAKE, None) == -1
    assert lib.lora_block8_decode(FAKE, 1, FAKE + 1, 5, FAKE, None) == -4
    assert lib.lora_block8_decode(None, 1, None, 0, None, None) == 0


def test_binding_refusals():
    A, B, s = torch.zeros(2, 16, 64).bfloat16(), torch.zeros(2, 32, 16).bfloat16(), torch.ones(2)
    wpg.AdapterBank(A, B, s)
    for bad in ((A[0], B, s), (A.transpose(1, 2), B, s), (A, B.float(), s), (A, B, s.double()), (A, B[:1], s),
                (A[:, :8].contiguous(), B, s)):
        with pytest.raises(ValueError):
            wpg.AdapterBank(*bad)
    bank, X = wpg.AdapterBank(A, B, s), torch.zeros(3, 64).bfloat16()
    for slot, rs in ((torch.zeros(3, dtype=torch.int64), None), (torch.zeros(4, dtype=torch.int32), None),
                     (torch.zeros(6, dtype=torch.int32)[::2], None), (torch.zeros(3, dtype=torch.int32), torch.zeros(2))):
        with pytest.raises(ValueError):
            wpg.lora_linear_fwd_multi(X, None, None, bank, slot, row_scale=rs)
    with pytest.raises(ValueError):
        wpg.lora_norm_fwd(torch.zeros(3, 8), torch.zeros(16)[::2])
    with pytest.raises(ValueError):
        wpg.lora_norm_bwd(torch.zeros(3, 8), torch.zeros(3, 8), None, torch.zeros(3))
    p, z = [torch.zeros(300)], [torch.zeros(300)]
    b8 = [wpg.Block8.zeros(300, True, "cpu")]
    for m, v in ((z, []), (b8, z), ([torch.zeros(299)], z), ([torch.zeros(300).double()], z), (b8, b8)):
        with pytest.raises(ValueError):
            wpg.lora_adamw_plan(p, m, v)
    with pytest.raises(ValueError):
        wpg.lora_block8_decode(torch.zeros(300, dtype=torch.int32), torch.zeros(2))


# --------------------------------------------------------------- the 64-bit definitions themselves
def test_norm_gradient_formula_against_differences():
    rng = np.random.default_rng(0)
    for layer in (True, False):
        x, dy, w = rng.standard_normal((3, 7)), rng.standard_normal((3, 7)), rng.standard_normal(7)
        _, mu, r = on.forward(x, w, None, 1e-3, layer)
        dx, dw, db = on.backward(dy, x, w, mu, r, layer)
        f = lambda x, w, b: (on.forward(x, w, b, 1e-3, layer)[0] * dy).sum()  # noqa: E731
        h = 1e-6
        for i in np.ndindex(3, 7):
            e = np.zeros((3, 7))
            e[i] = h
            assert abs((f(x + e, w, 0) - f(x - e, w, 0)) / (2 * h) - dx[i]) < 1e-7
        for j in range(7):
            e = np.zeros(7)
            e[j] = h
            assert abs((f(x, w + e, 0) - f(x, w - e, 0)) / (2 * h) - dw[j]) < 1e-7
            assert abs((f(x, w, e) - f(x, w, -e)) / (2 * h) - db[j]) < 1e-7


def test_adamw_first_step_and_codes():
    # one step from zero moments moves by lr against the gradient's sign (eps aside), after the decay
    p, m, v = oa.step(np.array([2.0, -1.0]), np.array([0.5, -3.0]), np.zeros(2), np.zeros(2), 0.1, 0.9, 0.999, 0.0, 0.5, 1)
    assert np.allclose(p, [2.0 * 0.95 - 0.1, -0.95 + 0.1]) and np.allclose(m, [0.05, -0.3])
    # each value's code is its nearest in the root's domain, the scale exact, zero kept
    x = np.array([0.0, 1.0, -1.0, 0.25, -0.25, 1e-9, -(60 / 127) ** 2], np.float32)
    q, top = oa.encode(x, True)
    assert list(q) == [0, 127, -127, 64, -64, 0, -60] and top[0] == 1
    q, top = oa.encode(np.abs(x), False)
    assert list(q[:3]) == [0, 255, 255] and q[5] == 1
    for signed in (True, False):
        codes = np.arange(-127 if signed else 0, 128 if signed else 256)
        back, _ = oa.encode(oa.decode(np.pad(codes, (0, 1 if signed else 0)), np.array([3.7], np.float32), signed), signed)
        assert np.array_equal(back[:len(codes)].astype(int), codes)
