"""Arguments of the adapter-set calls that a kernel could not use: refused on the host, before any
pointer is passed on."""
import ctypes

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


# ------------------------------------------------------------------------------ handles keep their memory
def test_a_banks_tensors_cannot_be_exchanged():
    A, B, scale = torch.zeros(2, 16, 64).bfloat16(), torch.zeros(2, 32, 16).bfloat16(), torch.ones(2)
    bank = wpg.AdapterBank(A, B, scale)
    for name, value in (("A", A.clone()), ("B", B.clone()), ("scale", scale.clone()), ("n_groups", 2), ("out_features", 8)):
        with pytest.raises(AttributeError):
            setattr(bank, name, value)
    assert (bank.A is A and bank.B is B and bank.scale is scale) and (bank.n_groups, bank.out_features) == (1, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_a_plan_keeps_the_memory_it_updates(bits):
    n = 1 << 20
    p, g = torch.ones(n, device=DEV), torch.ones(n, device=DEV)
    if bits == 8:
        m, v = wpg.Block8.zeros(n, True, DEV), wpg.Block8.zeros(n, False, DEV)
    else:
        m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    plan = wpg.lora_adamw_plan([p], [m], [v])
    old = p.data_ptr()
    p.data = torch.full((n,), 5.0, device=DEV)
    if bits == 8:
        m.codes, v.codes = m.codes.clone(), v.codes.clone()
    else:
        m.data, v.data = m.clone(), v.clone()
    fresh = [torch.full((n,), 7.0, device=DEV) for _ in range(4)]
    small = [torch.full((n,), 7, dtype=torch.uint8, device=DEV) for _ in range(4)]
    assert all(t.data_ptr() != old for t in fresh)
    wpg.lora_adamw_step(plan, [g], 1e-3)
    torch.cuda.synchronize()
    assert bool((p == 5.0).all()) and all(bool((t == 7).all()) for t in fresh + small)


@pytest.mark.gpu
def test_a_bank_keeps_the_memory_it_reads():
    A, B = torch.randn(2, 16, 64, device=DEV).bfloat16(), torch.randn(2, 32, 16, device=DEV).bfloat16()
    scale, X = torch.ones(2, device=DEV), torch.randn(5, 64, device=DEV).bfloat16()
    slot = torch.tensor([0, 1, 0, -1, 1], dtype=torch.int32, device=DEV)
    bank = wpg.AdapterBank(A, B, scale)
    want = wpg.lora_linear_fwd_multi(X, None, None, bank, slot)
    scale.data, A.data, B.data = torch.zeros(2, device=DEV), torch.zeros_like(A), torch.zeros_like(B)
    fresh = [torch.full_like(t, float("nan")) for t in (A, B, scale) for _ in range(3)]
    assert torch.equal(wpg.lora_linear_fwd_multi(X, None, None, bank, slot), want) and len(fresh) == 9


# ------------------------------------------------------------------------------ the C calls
FAKE = 0x10000
BF, F32, NF4 = wpg.WP_BF16, wpg.WP_FP32, wpg.WP_NF4
ALIGN, SHAPE = -4, -2


def _m(rows, cols, dtype=BF, data=FAKE, absmax=None, ld=None):
    return wpg.WpMat(data, dtype, rows, cols, cols if ld is None else ld, absmax)


def _o(rows, cols, dtype=BF, data=FAKE, ld=None):
    return wpg.WpOut(data, dtype, rows, cols, cols if ld is None else ld)


def _r(x):
    return None if x is None else ctypes.byref(x)


def _multi(W=None, bias=None, scale=FAKE, slot=FAKE, row_scale=None):
    bank = wpg.WpBank(FAKE, FAKE, scale, BF, 4, 1, 16, 128, 256)
    return wpg.lib().lora_linear_fwd_multi(_r(_m(9, 128)), _r(W), _r(bias), _r(bank), slot, row_scale, 1.0, _r(_o(9, 256)),
                                           FAKE, 1 << 40, None)


def _norm_fwd(X=None, weight=None, bias=None, Y=None, stats=FAKE):
    return wpg.lib().lora_norm_fwd(_r(X or _m(5, 64)), _r(weight), _r(bias), 0, 1e-5, _r(Y or _o(5, 64)), stats, None)


def _norm_bwd(dY=None, X=None, weight=None, stats=FAKE, dX=None, dW=None, dB=None):
    return wpg.lib().lora_norm_bwd(_r(dY or _m(5, 64)), _r(X or _m(5, 64)), _r(weight), stats, 0, _r(dX or _o(5, 64)),
                                   _r(dW), _r(dB), FAKE, 1 << 30, None)


def test_pointers_off_their_elements_boundary_are_refused():
    assert _multi(bias=_m(1, 256, data=FAKE + 1)) == ALIGN and _multi(bias=_m(1, 256, F32, FAKE + 2)) == ALIGN
    assert _multi(scale=FAKE + 2) == ALIGN and _multi(slot=FAKE + 1) == ALIGN and _multi(row_scale=FAKE + 2) == ALIGN
    assert _multi(W=_m(256, 128, NF4, absmax=FAKE + 2)) == ALIGN
    assert _norm_fwd(X=_m(5, 64, data=FAKE + 1)) == ALIGN and _norm_fwd(Y=_o(5, 64, data=FAKE + 1)) == ALIGN
    assert _norm_fwd(X=_m(5, 64, F32, FAKE + 2), Y=_o(5, 64, F32)) == ALIGN
    assert _norm_fwd(weight=_m(1, 64, data=FAKE + 1)) == ALIGN and _norm_fwd(bias=_m(1, 64, F32, FAKE + 2)) == ALIGN
    assert _norm_fwd(stats=FAKE + 2) == ALIGN
    assert _norm_bwd(dY=_m(5, 64, data=FAKE + 1)) == ALIGN and _norm_bwd(X=_m(5, 64, data=FAKE + 1)) == ALIGN
    assert _norm_bwd(dX=_o(5, 64, data=FAKE + 1)) == ALIGN and _norm_bwd(weight=_m(1, 64, F32, FAKE + 2)) == ALIGN
    assert _norm_bwd(stats=FAKE + 2) == ALIGN
    assert _norm_bwd(dW=_o(1, 64, F32, FAKE + 2)) == ALIGN and _norm_bwd(dB=_o(1, 64, F32, FAKE + 1)) == ALIGN


def test_a_vector_in_several_pieces_is_refused():
    # as a matrix whose rows lie apart, or a column of one
    assert _multi(bias=_m(2, 128, ld=136)) == SHAPE and _multi(bias=_m(256, 1, F32, ld=4)) == SHAPE
    assert _norm_fwd(weight=_m(2, 32, ld=40)) == SHAPE and _norm_fwd(bias=_m(64, 1, ld=2)) == SHAPE
    assert _norm_bwd(weight=_m(4, 16, F32, ld=24)) == SHAPE
    assert _norm_bwd(dW=_o(2, 32, F32, ld=48)) == SHAPE and _norm_bwd(dB=_o(64, 1, F32, ld=3)) == SHAPE


@pytest.mark.gpu
def test_a_stacked_bias():
    X, W = torch.randn(5, 64, device=DEV).bfloat16(), torch.randn(32, 64, device=DEV).bfloat16()
    bank = wpg.AdapterBank(torch.zeros(1, 16, 64, device=DEV).bfloat16(), torch.zeros(1, 32, 8, device=DEV).bfloat16(),
                           torch.ones(1, device=DEV), 2)
    slot = torch.full((5,), -1, dtype=torch.int32, device=DEV)
    wide = torch.randn(2, 24, device=DEV)
    want = wpg.lora_linear_fwd_multi(X, W, wide[:, :16].reshape(-1), bank, slot)
    assert torch.equal(wpg.lora_linear_fwd_multi(X, W, wide[:, :16].contiguous(), bank, slot), want)
    for bias in (wide[:, :16], torch.randn(32, 3, device=DEV)[:, :1]):
        with pytest.raises(wpg.WeightPatchesError, match="SHAPE"):
            wpg.lora_linear_fwd_multi(X, W, bias, bank, slot)


# ------------------------------------------------------------------------------ workspace
def _workspace(rows, K, N, G, R, slots, dtype):
    W = None if dtype is None else _m(N, K, dtype, absmax=FAKE if dtype == NF4 else None)
    bank = wpg.WpBank(FAKE, FAKE, FAKE, BF, slots, G, R, K, N)
    return wpg.lib().lora_multi_workspace_size(_r(_m(rows, K)), _r(W), _r(bank))


@pytest.mark.parametrize("dtype", [BF, NF4, None])
@pytest.mark.parametrize("K,N,G,R,slots", [(4096, 28672, 2, 16, 16), (64, 8, 1, 8, 1), (1536, 4608, 3, 32, 8),
                                           (5120, 5120, 1, 16, 64), (14336, 4096, 1, 16, 8), (8960, 5128, 1, 64, 300),
                                           (65536, 1024, 1, 256, 4), (262144, 64, 1, 8, 2)])
def test_the_workspace_for_more_rows_holds_fewer(K, N, G, R, slots, dtype):
    sizes = [_workspace(T, K, N, G, R, slots, dtype) for T in list(range(1, 600)) + [2048, 32760]]
    assert sizes[0] > 0 and sizes == sorted(sizes)
    # and the call asks for no more than the size of its own rows
    bank = wpg.WpBank(FAKE, FAKE, FAKE, BF, slots, G, R, K, N)
    W = None if dtype is None else _m(N, K, dtype, absmax=FAKE if dtype == NF4 else None)
    for T in (1, 7, 16, 64, 65, 97, 128, 129, 200, 256, 257, 500):
        call = lambda nbytes: wpg.lib().lora_linear_fwd_multi(  # noqa: E731
            _r(_m(T, K)), _r(W), None, _r(bank), FAKE, None, 1.0, _r(_o(T, N)), FAKE + 4, nbytes, None)
        assert call(_workspace(T, K, N, G, R, slots, dtype)) == ALIGN       # (the workspace's own alignment: nothing runs)
        assert call(64) == -5


@pytest.mark.gpu
@pytest.mark.parametrize("K,N", [(512, 5136), (4096, 1024)])
@pytest.mark.parametrize("T", [1, 9, 40, 100, 128, 140])
def test_a_workspace_for_more_rows_gives_the_same_bits(T, K, N):
    g = torch.Generator(device=DEV).manual_seed(T)
    X = torch.randn(T, K, generator=g, device=DEV).bfloat16()
    W = wpg.NF4Weight(torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8),
                      torch.rand(N * K // 64, generator=g, device=DEV), N, K)
    bank = wpg.AdapterBank(torch.randn(3, 16, K, generator=g, device=DEV).bfloat16(),
                           torch.randn(3, N, 16, generator=g, device=DEV).bfloat16(), torch.ones(3, device=DEV))
    slot = torch.randint(-1, 3, (T,), generator=g, device=DEV, dtype=torch.int32)
    size = wpg.lora_multi_workspace_size(torch.empty(2048, K, dtype=torch.bfloat16, device=DEV), W, bank)
    want = wpg.lora_linear_fwd_multi(X, W, None, bank, slot)
    got = wpg.lora_linear_fwd_multi(X, W, None, bank, slot, workspace=torch.empty(size, dtype=torch.uint8, device=DEV))
    assert torch.equal(got, want)


# ------------------------------------------------------------------------------ sizes
def test_sizes_beyond_the_kernels_32_bit_indexes_are_refused():
    def multi(T, K, N):
        bank = wpg.WpBank(FAKE, FAKE, FAKE, BF, 1, 1, 8, K, N)
        return wpg.lib().lora_linear_fwd_multi(_r(_m(T, K)), _r(_m(N, K)), None, _r(bank), FAKE, None, 1.0,
                                               _r(_o(T, N)), FAKE, 16, None)
    # rows and columns are rounded up to tiles, K to the steps of a CTA's warps
    for T, K, N in ((2 ** 31 - 1, 8, 8), (2 ** 31 - 256, 8, 8), (1, 2 ** 31 - 8, 8), (1, 2 ** 30, 8), (1, 8, 2 ** 31 - 8)):
        assert multi(T, K, N) == -8, (T, K, N)
    assert multi(2 ** 31 - 513, 8, 8) == multi(1, 2 ** 30 - 8, 8) == multi(1, 8, 2 ** 31 - 520) == -5


def test_a_norm_takes_a_matrix():
    with pytest.raises(ValueError, match="T, C"):
        wpg.lora_norm_fwd(torch.zeros(64))
    with pytest.raises(ValueError, match="T, C"):
        wpg.lora_norm_bwd(torch.zeros(64), torch.zeros(64), None, torch.zeros(2, 1))


# ------------------------------------------------------------------------------ AdamW's arrays
def test_a_set_whose_arrays_overlap_is_refused():
    def init(*tensors):
        arr = (wpg.WpAdamWTensor * len(tensors))(*tensors)
        return wpg.lib().lora_adamw_plan_init(arr, len(tensors), FAKE, 1 << 30, _r(wpg.WpAdamWPlan()), None)

    def t(at, numel=1000, dtype=F32, bits=32, **kw):
        a = dict(param=at, master=None, m=at + 0x100000, v=at + 0x200000, ms=at + 0x300000, vs=at + 0x400000)
        a.update(kw)
        return wpg.WpAdamWTensor(a["param"], a["master"], a["m"], a["v"], a["ms"], a["vs"], numel, dtype, bits)

    a, far = 0x10000000, 0x20000000
    assert init(t(a), t(a)) == -1                                     # listed twice
    assert init(t(a), t(far), t(far + 0x800000, m=a + 0x100000)) == -1    # two tensors with one state
    assert init(t(a, v=a + 0x100000)) == -1 and init(t(a, m=a + 3996)) == -1     # within one tensor; its last element
    assert init(t(a, dtype=BF, master=a + 1996)) == -1
    assert init(t(a, bits=8, m=a + 4000, v=a + 4999)) == -1
    assert init(t(a, bits=8, ms=a + 0x200000)) == -1 and init(t(a, bits=8, ms=far, vs=far + 12)) == -1


@pytest.mark.gpu
def test_a_set_whose_arrays_only_touch():
    # neighbours in one buffer; a tensor without elements may lie anywhere
    buf, m, v = (torch.zeros(1002, device=DEV) for _ in range(3))
    buf[:] = 1.0
    cut = lambda x: [x[:500], x[500:500], x[500:501], x[501:]]  # noqa: E731
    plan = wpg.lora_adamw_plan(cut(buf), cut(m), cut(v))
    wpg.lora_adamw_step(plan, [torch.ones_like(x) for x in cut(buf)], 0.1, weight_decay=0.0)
    assert (buf - 0.9).abs().max() < 1e-6
    with pytest.raises(wpg.WeightPatchesError, match="INVALID"):
        wpg.lora_adamw_plan([buf, buf[:10]], [m, torch.zeros(10, device=DEV)], [v, torch.zeros(10, device=DEV)])


# ------------------------------------------------------------------------------ the one-adapter calls' bias
def test_a_layers_bias_in_several_pieces_is_refused():
    lib, X, W, Y = wpg.lib(), _m(9, 128), _m(256, 128), _o(9, 256)
    ads = (wpg.WpAdapter * 2)(*[wpg.WpAdapter(_m(16, 128), _m(128, 16), 16.0, 1.0, None, 0) for _ in range(2)])
    for bias in (_m(2, 128, ld=136), _m(256, 1, F32, ld=4)):
        assert lib.lora_linear_fwd(_r(X), _r(W), _r(bias), None, 0, 1.0, _r(Y), FAKE, 1 << 40, None) == SHAPE
        assert lib.lora_linear_fwd_grouped(_r(X), _r(W), _r(bias), 2, ads, 1.0, _r(Y), FAKE, 1 << 40, None) == SHAPE
        out = wpg.WpOut(bias.data, bias.dtype, bias.rows, bias.cols, bias.ld)
        assert lib.lora_merge(_r(W), _r(out), None, 0, 1.0, FAKE, 1 << 40, None) == SHAPE
