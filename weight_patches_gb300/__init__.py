"""weight_patches_gb300 -- the dynamic, unmerged LoRA linear on GB300 (sm_103a).

A thin ctypes binding over ``libweight_patches_gb300.so`` (C ABI in
``include/weight_patches.h``).  The functions here only marshal arguments: torch
tensors supply device memory and the current CUDA stream; every step of the
computation runs in the library's CUDA kernels.  There is no fallback: if the shared
library has not been built, importing it raises.

Entry points (same names as the C ABI):
    lora_linear_fwd          Y = X W^T + bias + sum_p s_p (X A_p^T) B_p^T
    lora_linear_fwd_grouped  stacked column groups, one adapter per group
    lora_linear_bwd          closed-form dX, dA, dB
    lora_linear_fwd_exact    the unfused bf16 chain (the "exact" tier), unit scales skipped or not
    lora_dense_patch         .diff / .diff_b (add) and .set_weight (replace), in place
    lora_linear_fwd_multi    one projection for rows of many adapters (an AdapterBank)
    lora_norm_fwd / _bwd     layer norm or RMS norm, and the gradients of x, weight, bias
    lora_adamw_plan / _step  one AdamW step over many tensors, 32- or 8-bit moments
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libweight_patches_gb300.so")

WP_BF16, WP_FP32, WP_NF4 = 0, 1, 2
WP_PATCH_ADD, WP_PATCH_SET = 0, 1
WP_OP_FWD, WP_OP_FWD_GROUPED, WP_OP_BWD, WP_OP_FWD_HOST, WP_OP_SWIGLU_FWD, WP_OP_MERGE, WP_OP_FWD_EXACT, WP_OP_NORM_BWD = range(8)
WP_NORM_LAYER, WP_NORM_RMS = 0, 1
STATUS = {0: "WP_OK", -1: "WP_ERR_INVALID", -2: "WP_ERR_SHAPE", -3: "WP_ERR_DTYPE",
          -4: "WP_ERR_ALIGN", -5: "WP_ERR_WORKSPACE", -6: "WP_ERR_CUDA", -7: "WP_ERR_TIMEOUT",
          -8: "WP_ERR_UNSUPPORTED"}


class WpMat(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("ld", ctypes.c_int64), ("absmax", ctypes.c_void_p)]


class WpOut(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("ld", ctypes.c_int64)]


class WpAdapter(ctypes.Structure):
    _fields_ = [("A", WpMat), ("B", WpMat), ("alpha", ctypes.c_double),
                ("strength", ctypes.c_double), ("bias_B", ctypes.c_void_p), ("bias_B_dtype", ctypes.c_int32)]


class WpBank(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("n_slots", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("in_", ctypes.c_int64), ("out", ctypes.c_int64)]


class WpAdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("master", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_absmax", ctypes.c_void_p), ("v_absmax", ctypes.c_void_p),
                ("numel", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("state_bits", ctypes.c_int32)]


class WpAdamWPlan(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("n_tensors", ctypes.c_int32), ("n_launches", ctypes.c_int32),
                ("unit_begin", ctypes.c_int64 * 17), ("launches_8bit", ctypes.c_uint32)]


class WpAdamWArgs(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("step", ctypes.c_int64), ("grad_scale_dev", ctypes.c_void_p)]


class WeightPatchesError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        lib = _load()
        msg = lib.lora_status_string(status).decode()
        cuda = lib.lora_last_cuda_error().decode()
        super().__init__(f"{where}: {STATUS.get(status, status)} ({msg}){' / ' + cuda if cuda else ''}")


_LIB = None


def _load():
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()'"
            " or python weight_patches_gb300/build.py)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, D, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t
    pm, po, pa = ctypes.POINTER(WpMat), ctypes.POINTER(WpOut), ctypes.POINTER(WpAdapter)
    lib.lora_linear_fwd.argtypes = [pm, pm, pm, pa, I32, D, po, P, SZ, P]
    lib.lora_linear_fwd_grouped.argtypes = [pm, pm, pm, I32, pa, D, po, P, SZ, P]
    lib.lora_linear_fwd_noalloc.argtypes = [pm, pm, pm, pa, I32, D, po, P]
    lib.lora_linear_fwd_host.argtypes = [pm, pm, pm, I32, pa, I32, D, po, P, SZ, P]
    lib.lora_linear_fwd_exact.argtypes = [pm, pm, pm, I32, pa, I32, D, I32, po, P, SZ, P]
    lib.lora_linear_bwd.argtypes = [pm, pm, pm, I32, pa, D, po, po, po, P, SZ, P]
    lib.lora_swiglu_fwd.argtypes = [pm, pm, pm, pa, D, po, po, P, SZ, P]
    lib.lora_merge.argtypes = [pm, po, pa, I32, D, P, SZ, P]
    lib.lora_merge_seeded.argtypes = [pm, po, pa, I32, D, ctypes.c_uint64, P, SZ, P]
    lib.lora_swiglu_bwd.argtypes = [pm, pm, po, po, P]
    lib.lora_dense_patch.argtypes = [P, I32, I64, P, I32, I64, I32, D, P]
    pb = ctypes.POINTER(WpBank)
    pt, pp = ctypes.POINTER(WpAdamWTensor), ctypes.POINTER(WpAdamWPlan)
    # the calls of decode and training steps take their structs as packed bytes (_pmat, _pout)
    lib.lora_linear_fwd_multi.argtypes = [P, P, P, P, P, P, D, P, P, SZ, P]
    lib.lora_multi_workspace_size.argtypes = [pm, pm, pb]
    lib.lora_multi_workspace_size.restype = SZ
    lib.lora_norm_fwd.argtypes = [P, P, P, I32, D, P, P, P]
    lib.lora_norm_bwd.argtypes = [P, P, P, P, I32, P, P, P, P, SZ, P]
    lib.lora_adamw_plan_size.argtypes = [pt, I32]
    lib.lora_adamw_plan_size.restype = SZ
    lib.lora_adamw_plan_init.argtypes = [pt, I32, P, SZ, pp, P]
    lib.lora_adamw_step.argtypes = [P, P, I32, P, P]
    lib.lora_block8_decode.argtypes = [P, I32, P, I64, P, P]
    lib.lora_workspace_size.argtypes = [I32, pm, pm, pa, I32]
    lib.lora_workspace_size.restype = SZ
    lib.lora_status_string.argtypes = [ctypes.c_int]
    lib.lora_status_string.restype = ctypes.c_char_p
    lib.lora_device_status.argtypes = [I32]
    lib.lora_set_wait_limit.argtypes = [ctypes.c_uint64]
    lib.lora_debug_hold_flags.argtypes = [I32]
    lib.lora_nf4_codebook.argtypes = [ctypes.POINTER(ctypes.c_float)]
    lib.lora_nf4_codebook.restype = None
    lib.lora_last_cuda_error.restype = ctypes.c_char_p
    for name in ("lora_linear_fwd", "lora_linear_fwd_grouped", "lora_linear_bwd", "lora_dense_patch",
                 "lora_device_status", "lora_linear_fwd_noalloc", "lora_linear_fwd_host",
                 "lora_linear_fwd_exact", "lora_set_wait_limit", "lora_debug_hold_flags",
                 "lora_linear_fwd_multi", "lora_norm_fwd", "lora_norm_bwd", "lora_adamw_plan_init",
                 "lora_adamw_step", "lora_block8_decode"):
        getattr(lib, name).restype = ctypes.c_int
    _LIB = lib
    return lib


def lib():
    """The loaded shared library (ctypes.CDLL)."""
    return _load()


# ------------------------------------------------------------------------- marshalling
@dataclass
class NF4Weight:
    """A 4-bit NormalFloat weight [rows, cols]: ``packed`` uint8 [rows, cols // 2] (element
    2k in the high nibble of byte k), ``absmax`` fp32 [rows * cols // 64]."""

    packed: torch.Tensor
    absmax: torch.Tensor
    rows: int
    cols: int


@dataclass
class Adapter:
    """One low-rank patch: A [r, in], B [out, r] (bf16, or fp32 for an FP32 adapter), and the
    optional legacy ``bias_B`` [out] (bf16 or fp32) older adapters carry as lora_B.bias: the
    forwards add s * bias_B to the patch's output columns, ``lora_merge`` adds it to the
    module's bias."""

    A: torch.Tensor
    B: torch.Tensor
    alpha: float
    strength: float = 1.0
    bias_B: Optional[torch.Tensor] = None


_DT = {torch.bfloat16: WP_BF16, torch.float32: WP_FP32}


def _mat(t) -> Optional[WpMat]:
    if t is None:
        return None
    if isinstance(t, NF4Weight):
        if not (t.packed.is_contiguous() and t.absmax.is_contiguous()):
            raise ValueError("NF4Weight tensors must be contiguous")
        return WpMat(t.packed.data_ptr(), WP_NF4, t.rows, t.cols, t.cols, t.absmax.data_ptr())
    if t.dim() == 1:
        return WpMat(t.data_ptr(), _DT[t.dtype], 1, t.shape[0], t.shape[0], None)
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D row-major tensor (stride(1) == 1)")
    return WpMat(t.data_ptr(), _DT[t.dtype], t.shape[0], t.shape[1], t.stride(0), None)


def _out(t: torch.Tensor) -> WpOut:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D row-major output tensor")
    return WpOut(t.data_ptr(), _DT[t.dtype], t.shape[0], t.shape[1], t.stride(0))


def _adapters(adapters: Sequence[Adapter]):
    arr = (WpAdapter * max(1, len(adapters)))()
    for i, a in enumerate(adapters):
        vb = getattr(a, "bias_B", None)
        if vb is not None and not vb.is_contiguous():
            raise ValueError("bias_B must be contiguous")
        arr[i] = WpAdapter(_mat(a.A), _mat(a.B), float(a.alpha), float(a.strength),
                           vb.data_ptr() if vb is not None else None,
                           _DT[vb.dtype] if vb is not None else WP_BF16)
    return arr


def _ref(m):
    return ctypes.byref(m) if m is not None else None


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# Marshalling of the calls whose kernels take microseconds: a struct as packed bytes costs a tenth
# of a ctypes.Structure, the raw stream handle a twentieth of a Stream object.
_pack_mat = struct.Struct("@PiqqqP").pack        # wp_mat
_pack_adamw = struct.Struct("@ddddddqP").pack    # wp_adamw_args
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _pmat(t) -> Optional[bytes]:
    if t is None:
        return None
    if isinstance(t, NF4Weight):
        return bytes(_mat(t))
    shape = t.shape
    if len(shape) == 2:
        ld, one = t.stride()
        if one != 1 and shape[1] != 1:
            raise ValueError("expected a 2-D row-major tensor (stride(1) == 1)")
        return _pack_mat(t.data_ptr(), _DT[t.dtype], shape[0], shape[1], ld if shape[0] > 1 else max(ld, shape[1]), 0)
    if len(shape) != 1 or not t.is_contiguous():
        raise ValueError("expected a row-major matrix or a contiguous vector")
    return _pack_mat(t.data_ptr(), _DT[t.dtype], 1, shape[0], shape[0], 0)


def _pout(t: torch.Tensor) -> bytes:
    return _pmat(t)[:40]                          # wp_out: wp_mat without its last pointer


def _one_device(call: str, first: torch.Tensor, *others) -> int:
    """The index of the CUDA device that all of a call's tensors lie on (None: an argument not given).
    A kernel would read a host pointer as its own memory."""
    index = first.get_device()
    for t in others:
        if t is None:
            continue
        if isinstance(t, NF4Weight):
            if t.absmax.get_device() != index:
                break
            t = t.packed
        if t.get_device() != index:
            break
    else:
        if index >= 0:
            return index
    raise ValueError(f"{call}: its tensors must be on one CUDA device")


def _check(status: int, where: str):
    if status != 0:
        raise WeightPatchesError(status, where)


def _workspace(op, xm, wm, arr, n, device, workspace):
    need = _load().lora_workspace_size(op, ctypes.byref(xm), _ref(wm), arr, n)
    if need == 0:
        return None, 0
    if workspace is not None and workspace.numel() * workspace.element_size() >= need:
        return workspace, need
    return torch.empty(need, dtype=torch.uint8, device=device), need


def lora_workspace_size(op: int, X, W, adapters: Sequence[Adapter]) -> int:
    xm, wm, arr = _mat(X), _mat(W), _adapters(adapters)
    return _load().lora_workspace_size(op, _ref(xm), _ref(wm), arr, len(adapters))


def _out_features(X, W, adapters):
    if W is not None:
        return W.rows if isinstance(W, NF4Weight) else W.shape[0]
    return adapters[0].B.shape[0]


def lora_linear_fwd(X: torch.Tensor, W, bias: Optional[torch.Tensor], adapters: Sequence[Adapter],
                    request_scale: float = 1.0, out: Optional[torch.Tensor] = None,
                    out_dtype: torch.dtype = torch.bfloat16,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = X W^T + bias + sum_p s_p (X A_p^T) B_p^T with s_p = alpha/r * strength * request_scale."""
    if out is None:
        out = torch.empty(X.shape[0], _out_features(X, W, adapters), dtype=out_dtype, device=X.device)
    xm, wm, bm, arr, ym = _mat(X), _mat(W), _mat(bias), _adapters(adapters), _out(out)
    ws, nbytes = _workspace(WP_OP_FWD, xm, wm, arr, len(adapters), X.device, workspace)
    st = _load().lora_linear_fwd(ctypes.byref(xm), _ref(wm), _ref(bm), arr, len(adapters),
                                 float(request_scale), ctypes.byref(ym),
                                 ws.data_ptr() if ws is not None else None, nbytes, _stream(X.device))
    _check(st, "lora_linear_fwd")
    return out


def lora_linear_fwd_grouped(X: torch.Tensor, W_stacked, bias: Optional[torch.Tensor],
                            adapters: Sequence[Adapter], request_scale: float = 1.0,
                            out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Stacked column groups: group g of the output gets X W_g^T + bias_g + s_g (X A_g^T) B_g^T."""
    n = W_stacked.rows if isinstance(W_stacked, NF4Weight) else W_stacked.shape[0]
    if out is None:
        out = torch.empty(X.shape[0], n, dtype=out_dtype, device=X.device)
    xm, wm, bm, arr, ym = _mat(X), _mat(W_stacked), _mat(bias), _adapters(adapters), _out(out)
    ws, nbytes = _workspace(WP_OP_FWD_GROUPED, xm, wm, arr, len(adapters), X.device, workspace)
    st = _load().lora_linear_fwd_grouped(ctypes.byref(xm), ctypes.byref(wm), _ref(bm), len(adapters),
                                         arr, float(request_scale), ctypes.byref(ym),
                                         ws.data_ptr() if ws is not None else None, nbytes,
                                         _stream(X.device))
    _check(st, "lora_linear_fwd_grouped")
    return out


def lora_merge(W, adapters: Sequence[Adapter], scale: float = 1.0, workspace: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, rounding_seed: Optional[int] = None):
    """Bake the adapters into W in place: W <- W + sum_p s_p B_p A_p (s_p = alpha/r * strength
    * scale), accumulated in fp32 and rounded once; a 4-bit ``NF4Weight`` is requantised,
    round to nearest, or with ``rounding_seed`` (an unsigned 64-bit integer) stochastically
    (``lora_merge_seeded``).  Adapters with a legacy ``bias_B`` also update ``bias`` in place
    (bias <- bias + sum_p s_p bias_B_p, one rounding); the call fails before writing anything
    when such an adapter meets ``bias=None``.  Returns W."""
    wm, arr = _mat(W), _adapters(adapters)
    bo = None
    if bias is not None:
        if not bias.is_contiguous():
            raise ValueError("bias must be contiguous")
        bo = WpOut(bias.data_ptr(), _DT[bias.dtype], 1, bias.numel(), bias.numel())
    device = W.packed.device if isinstance(W, NF4Weight) else W.device
    need = _load().lora_workspace_size(WP_OP_MERGE, None, ctypes.byref(wm), arr, len(adapters))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    nbytes = workspace.numel() if workspace is not None else 0
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    if rounding_seed is None:
        st = _load().lora_merge(ctypes.byref(wm), _ref(bo), arr, len(adapters), float(scale), ws_ptr, nbytes,
                                _stream(device))
        _check(st, "lora_merge")
    else:
        seed = int(rounding_seed)
        if not 0 <= seed < 1 << 64:
            raise ValueError("rounding_seed must be an unsigned 64-bit integer")
        st = _load().lora_merge_seeded(ctypes.byref(wm), _ref(bo), arr, len(adapters), float(scale), seed, ws_ptr,
                                       nbytes, _stream(device))
        _check(st, "lora_merge_seeded")
    return W


def lora_swiglu_fwd(X: torch.Tensor, W_gate_up, bias: Optional[torch.Tensor], adapters: Sequence[Adapter],
                    request_scale: float = 1.0, out: Optional[torch.Tensor] = None,
                    eg: Optional[torch.Tensor] = None, save_eg: bool = False,
                    workspace: Optional[torch.Tensor] = None):
    """SwiGLU front half: h = silu(e) g with e, g the gate and up LoRA linears of the stacked
    ``W_gate_up`` ([2F, in]; ``adapters`` = [gate, up]).  Returns h, or (h, eg) when
    ``save_eg`` or ``eg`` is given (eg = e | g, [T, 2F], what the backward needs)."""
    n2 = W_gate_up.rows if isinstance(W_gate_up, NF4Weight) else W_gate_up.shape[0]
    if out is None:
        out = torch.empty(X.shape[0], n2 // 2, dtype=torch.bfloat16, device=X.device)
    if eg is None and save_eg:
        eg = torch.empty(X.shape[0], n2, dtype=torch.bfloat16, device=X.device)
    xm, wm, bm, arr, hm = _mat(X), _mat(W_gate_up), _mat(bias), _adapters(adapters), _out(out)
    egm = _out(eg) if eg is not None else None
    ws, nbytes = _workspace(WP_OP_SWIGLU_FWD, xm, wm, arr, len(adapters), X.device, workspace)
    st = _load().lora_swiglu_fwd(ctypes.byref(xm), ctypes.byref(wm), _ref(bm), arr, float(request_scale),
                                 ctypes.byref(hm), _ref(egm), ws.data_ptr() if ws is not None else None,
                                 nbytes, _stream(X.device))
    _check(st, "lora_swiglu_fwd")
    return (out, eg) if eg is not None else out


def lora_swiglu_bwd(dH: torch.Tensor, eg: torch.Tensor, deg: Optional[torch.Tensor] = None,
                    h: Optional[torch.Tensor] = None, want_h: bool = False):
    """SwiGLU backward: from the gradient at h and the saved e | g, de | dg ([T, 2F], the
    stacked gate/up output gradient); with ``want_h`` (or ``h``) also h recomputed.
    Returns deg, or (deg, h)."""
    if deg is None:
        deg = torch.empty_like(eg)
    if h is None and want_h:
        h = torch.empty_like(dH)
    hm = _out(h) if h is not None else None
    st = _load().lora_swiglu_bwd(ctypes.byref(_mat(dH)), ctypes.byref(_mat(eg)), ctypes.byref(_out(deg)),
                                 _ref(hm), _stream(dH.device))
    _check(st, "lora_swiglu_bwd")
    return (deg, h) if h is not None else deg


def lora_linear_fwd_host(X_host: torch.Tensor, W, bias: Optional[torch.Tensor], adapters: Sequence[Adapter],
                         request_scale: float = 1.0, out: Optional[torch.Tensor] = None,
                         out_dtype: torch.dtype = torch.bfloat16, grouped: bool = False,
                         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The forward with X and the result in host memory (pin both for the copies to overlap
    the compute): rows go through the device in chunks, copies and kernels overlapped.
    ``grouped`` selects the stacked column-group form (one adapter per group)."""
    if isinstance(W, NF4Weight):
        device, n = W.packed.device, W.rows
    elif W is not None:
        device, n = W.device, W.shape[0]
    else:
        device, n = adapters[0].A.device, adapters[0].B.shape[0]
    if out is None:
        out = torch.empty(X_host.shape[0], n, dtype=out_dtype, pin_memory=True)
    xm, wm, bm, arr, ym = _mat(X_host), _mat(W), _mat(bias), _adapters(adapters), _out(out)
    ws, nbytes = _workspace(WP_OP_FWD_HOST, xm, wm, arr, len(adapters), device, workspace)
    st = _load().lora_linear_fwd_host(ctypes.byref(xm), _ref(wm), _ref(bm), len(adapters) if grouped else 0,
                                      arr, len(adapters), float(request_scale), ctypes.byref(ym),
                                      ws.data_ptr() if ws is not None else None, nbytes, _stream(device))
    _check(st, "lora_linear_fwd_host")
    return out


def lora_linear_fwd_exact(X: torch.Tensor, W, bias: Optional[torch.Tensor], adapters: Sequence[Adapter],
                          request_scale: float = 1.0, skip_unit_scales: bool = True, grouped: bool = False,
                          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The unfused bf16 chain (base, X A^T, then B^T, one rounded multiplication per scale, the
    add), the exact tier when ``skip_unit_scales``; ``grouped``: one adapter per column group."""
    n = W.rows if isinstance(W, NF4Weight) else W.shape[0]
    if out is None:
        out = torch.empty(X.shape[0], n, dtype=torch.bfloat16, device=X.device)
    xm, wm, bm, arr, ym = _mat(X), _mat(W), _mat(bias), _adapters(adapters), _out(out)
    ws, nbytes = _workspace(WP_OP_FWD_EXACT, xm, wm, arr, len(adapters), X.device, workspace)
    st = _load().lora_linear_fwd_exact(ctypes.byref(xm), ctypes.byref(wm), _ref(bm), len(adapters) if grouped else 0,
                                       arr, len(adapters), float(request_scale), 1 if skip_unit_scales else 0,
                                       ctypes.byref(ym), ws.data_ptr() if ws is not None else None, nbytes,
                                       _stream(X.device))
    _check(st, "lora_linear_fwd_exact")
    return out


def lora_linear_bwd(X: torch.Tensor, W, dY: torch.Tensor, adapters: Sequence[Adapter],
                    request_scale: float = 1.0, need_dX: bool = True,
                    dX_dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None):
    """Closed-form (dX, [dA_g], [dB_g]) of Y = X W_g^T + s_g (X A_g^T) B_g^T over len(adapters) groups."""
    G = len(adapters)
    dX = torch.empty_like(X, dtype=dX_dtype) if need_dX else None
    dA = [torch.empty(a.A.shape, dtype=torch.float32, device=X.device) for a in adapters]
    dB = [torch.empty(a.B.shape, dtype=torch.float32, device=X.device) for a in adapters]
    xm, wm, dym, arr = _mat(X), _mat(W), _mat(dY), _adapters(adapters)
    dxo = _out(dX) if dX is not None else None
    dao = (WpOut * G)(*[_out(t) for t in dA])
    dbo = (WpOut * G)(*[_out(t) for t in dB])
    ws, nbytes = _workspace(WP_OP_BWD, xm, wm, arr, G, X.device, workspace)
    st = _load().lora_linear_bwd(ctypes.byref(xm), ctypes.byref(wm), ctypes.byref(dym), G, arr,
                                 float(request_scale), _ref(dxo), dao, dbo,
                                 ws.data_ptr() if ws is not None else None, nbytes, _stream(X.device))
    _check(st, "lora_linear_bwd")
    return dX, dA, dB


def lora_dense_patch(param: torch.Tensor, payload: torch.Tensor, kind: int, strength: float = 1.0) -> torch.Tensor:
    """Apply a dense payload to ``param`` in place (.diff/.diff_b: kind=WP_PATCH_ADD,
    .set_weight: kind=WP_PATCH_SET) and return it."""
    if not (param.is_contiguous() and payload.is_contiguous()):
        raise ValueError("dense patch tensors must be contiguous")
    st = _load().lora_dense_patch(param.data_ptr(), _DT[param.dtype], param.numel(), payload.data_ptr(),
                                  _DT[payload.dtype], payload.numel(), int(kind), float(strength),
                                  _stream(param.device))
    _check(st, "lora_dense_patch")
    return param


# ------------------------------------------------------------------- adapters of many requests
class AdapterBank:
    """The adapters of one layer, one per slot, each padded with zeros to one rank:
    ``A`` [slots, n_groups * rank, in] and ``B`` [slots, out, rank] bf16, ``scale`` [slots] fp32
    (alpha / r * strength of each adapter), all contiguous on one device.  The tensors may be
    rewritten in place (an adapter loaded into its slot) between calls; they cannot be exchanged for
    others: build another bank."""

    def __init__(self, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor, n_groups: int = 1):
        if A.dim() != 3 or B.dim() != 3 or scale.dim() != 1:
            raise ValueError("AdapterBank: A [slots, groups * rank, in], B [slots, out, rank], scale [slots]")
        if not (A.is_contiguous() and B.is_contiguous() and scale.is_contiguous()):
            raise ValueError("AdapterBank tensors must be contiguous")
        if A.dtype not in _DT or B.dtype != A.dtype or scale.dtype != torch.float32:
            raise ValueError("AdapterBank: A and B of one dtype, scale float32")
        if not (A.shape[0] == B.shape[0] == scale.shape[0] and A.shape[1] == n_groups * B.shape[2]):
            raise ValueError("AdapterBank: the shapes of A, B and scale disagree")
        if not A.device == B.device == scale.device:
            raise ValueError("AdapterBank tensors must be on one device")
        self._A, self._B, self._scale, self._n_groups = A, B, scale, n_groups
        # the memory at the packed addresses lives as long as the bank does
        self._kept = A.untyped_storage(), B.untyped_storage(), scale.untyped_storage()
        self._c = WpBank(A.data_ptr(), B.data_ptr(), scale.data_ptr(), _DT[A.dtype], A.shape[0], n_groups,
                         B.shape[2], A.shape[2], B.shape[1])
        self._packed = bytes(self._c)

    A = property(lambda self: self._A)
    B = property(lambda self: self._B)
    scale = property(lambda self: self._scale)
    n_groups = property(lambda self: self._n_groups)
    out_features = property(lambda self: self._c.out)


def lora_multi_workspace_size(X: torch.Tensor, W, bank: AdapterBank) -> int:
    return _load().lora_multi_workspace_size(_ref(_mat(X)), _ref(_mat(W)), ctypes.byref(bank._c))


def lora_linear_fwd_multi(X: torch.Tensor, W, bias: Optional[torch.Tensor], bank: AdapterBank, slot: torch.Tensor,
                          row_scale: Optional[torch.Tensor] = None, request_scale: float = 1.0,
                          out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                          workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y[t] = X[t] W^T + bias + s_t (X[t] A_a^T) B_a^T with a = slot[t] (int32; a value outside the
    bank, -1 by convention, uses no adapter) and s_t = bank.scale[a] * row_scale[t] * request_scale;
    with ``bank.n_groups`` > 1, per stacked column group.  W bf16, ``NF4Weight`` or None."""
    T = X.shape[0]
    if slot.dtype is not torch.int32 or slot.numel() != T or not slot.is_contiguous():
        raise ValueError("slot must be a contiguous int32 tensor with one entry per row of X")
    if row_scale is not None and (row_scale.dtype is not torch.float32 or row_scale.numel() != T
                                  or not row_scale.is_contiguous()):
        raise ValueError("row_scale must be a contiguous float32 tensor with one entry per row of X")
    device = _one_device("lora_linear_fwd_multi", X, W, bias, bank._A, slot, row_scale, out, workspace)
    if out is None:
        out = torch.empty(T, bank.out_features, dtype=out_dtype, device=X.device)
    lib = _load()
    if workspace is None:
        workspace = torch.empty(max(lora_multi_workspace_size(X, W, bank), 1), dtype=torch.uint8, device=X.device)
    st = lib.lora_linear_fwd_multi(_pmat(X), _pmat(W), _pmat(bias), bank._packed, slot.data_ptr(),
                                   None if row_scale is None else row_scale.data_ptr(), request_scale, _pout(out),
                                   workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                   _raw_stream(device))
    if st:
        _check(st, "lora_linear_fwd_multi")
    return out


# ----------------------------------------------------------------------------------- norms
def lora_norm_fwd(X: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  eps: float = 1e-5, kind: int = WP_NORM_LAYER, out: Optional[torch.Tensor] = None,
                  stats: Optional[torch.Tensor] = None):
    """y = (x - mu) r w + b over the rows of X [T, C] (kind ``WP_NORM_RMS``: mu = 0).  Returns
    (y, stats), stats [2, T] fp32 holding mu and r for ``lora_norm_bwd``."""
    _check_rows(X)
    device = _one_device("lora_norm_fwd", X, weight, bias, out, stats)
    if out is None:
        out = torch.empty(X.shape, dtype=X.dtype, device=X.device)
    if stats is None:
        stats = torch.empty(2, X.shape[0], dtype=torch.float32, device=X.device)
    else:
        _check_stats(stats, X.shape[0])
    st = _load().lora_norm_fwd(_pmat(X), _pvec(weight), _pvec(bias), kind, eps, _pout(out), stats.data_ptr(),
                               _raw_stream(device))
    if st:
        _check(st, "lora_norm_fwd")
    return out, stats


def lora_norm_bwd_workspace_size(X: torch.Tensor) -> int:
    return _load().lora_workspace_size(WP_OP_NORM_BWD, _ref(_mat(X)), None, None, 0)


def lora_norm_bwd(dY: torch.Tensor, X: torch.Tensor, weight: Optional[torch.Tensor], stats: torch.Tensor,
                  kind: int = WP_NORM_LAYER, need_dx: bool = True, need_dw: bool = True, need_db: bool = True,
                  workspace: Optional[torch.Tensor] = None):
    """(dX, dW, dB) of ``lora_norm_fwd`` from its stats; dW and dB fp32 [C], None where not asked for."""
    _check_rows(X)
    T, C = X.shape
    _check_stats(stats, T)
    device = _one_device("lora_norm_bwd", X, dY, weight, stats, workspace)
    dev = X.device
    dx = torch.empty(T, C, dtype=X.dtype, device=dev) if need_dx else None
    dw = torch.empty(C, dtype=torch.float32, device=dev) if need_dw else None
    db = torch.empty(C, dtype=torch.float32, device=dev) if need_db else None
    if workspace is None and (need_dw or need_db):
        workspace = torch.empty(max(lora_norm_bwd_workspace_size(X), 1), dtype=torch.uint8, device=dev)
    st = _load().lora_norm_bwd(_pmat(dY), _pmat(X), _pvec(weight), stats.data_ptr(), kind,
                               None if dx is None else _pout(dx), None if dw is None else _pout(dw),
                               None if db is None else _pout(db), None if workspace is None else workspace.data_ptr(),
                               0 if workspace is None else workspace.numel() * workspace.element_size(),
                               _raw_stream(device))
    if st:
        _check(st, "lora_norm_bwd")
    return dx, dw, db


def _pvec(t: Optional[torch.Tensor]) -> Optional[bytes]:
    if t is not None and t.dim() != 1:
        raise ValueError("weight and bias of a norm must be contiguous vectors")
    return _pmat(t)


def _check_rows(X: torch.Tensor):
    if X.dim() != 2:
        raise ValueError("a norm's X must be a matrix [T, C]")


def _check_stats(stats: torch.Tensor, T: int):
    if stats.dtype != torch.float32 or stats.numel() != 2 * T or not stats.is_contiguous():
        raise ValueError("stats must be a contiguous float32 tensor [2, T]")


# ----------------------------------------------------------------------------------- AdamW
@dataclass
class Block8:
    """8-bit moments of one tensor: ``codes`` int8 (first moment) or uint8 (second), flat, and
    ``absmax`` fp32, one per 256 elements.  Zeros are the initial state."""

    codes: torch.Tensor
    absmax: torch.Tensor

    @staticmethod
    def zeros(numel: int, signed: bool, device) -> "Block8":
        return Block8(torch.zeros(numel, dtype=torch.int8 if signed else torch.uint8, device=device),
                      torch.zeros((numel + 255) // 256, dtype=torch.float32, device=device))


class AdamWPlan:
    """A prepared set of tensors (``lora_adamw_plan``); keeps their memory and the device table."""

    def __init__(self, c: WpAdamWPlan, table: torch.Tensor, kept, numels):
        self._table, self._kept, self._numels = table, kept, numels
        self._packed = bytes(c)
        self._pack_ptrs = struct.Struct(f"@{len(numels)}P").pack


def lora_adamw_plan(params: Sequence[torch.Tensor], m: Sequence, v: Sequence,
                    masters: Optional[Sequence[Optional[torch.Tensor]]] = None) -> AdamWPlan:
    """Prepare ``lora_adamw_step`` over ``params`` (bf16 or fp32, contiguous), their moments (fp32
    tensors, or ``Block8``) and, for bf16 parameters, optional fp32 masters that the step updates in
    their place.  The plan keeps and updates the memory that these tensors have now: build it again when
    one is given other memory (``p.data = ...``, ``Block8.codes = ...``)."""
    n = len(params)
    masters = list(masters) if masters is not None else [None] * n
    if not (n > 0 and n == len(m) == len(v) == len(masters)):
        raise ValueError("lora_adamw_plan: params, m, v and masters must be lists of one length")
    arr = (WpAdamWTensor * n)()
    kept = []                                         # the memory behind the table's addresses
    device = params[0].device
    for i, (p, mi, vi, ma) in enumerate(zip(params, m, v, masters)):
        numel, eight = p.numel(), isinstance(mi, Block8)
        if isinstance(vi, Block8) != eight:
            raise ValueError("lora_adamw_plan: m and v of one tensor are held alike")
        if eight:
            parts = [(mi.codes, torch.int8, numel), (vi.codes, torch.uint8, numel),
                     (mi.absmax, torch.float32, (numel + 255) // 256), (vi.absmax, torch.float32, (numel + 255) // 256)]
        else:
            parts = [(mi, torch.float32, numel), (vi, torch.float32, numel)]
        if ma is not None:
            parts.append((ma, torch.float32, numel))
        for t, dt, count in parts:
            if t.dtype != dt or t.numel() != count or not t.is_contiguous() or t.device != device:
                raise ValueError(f"lora_adamw_plan: tensor {i}: a state of the wrong dtype, size, layout or device")
        if p.dtype not in _DT or not p.is_contiguous() or p.device != device:
            raise ValueError(f"lora_adamw_plan: parameter {i} must be contiguous bf16 or fp32 on {device}")
        kept += [p.untyped_storage()] + [t.untyped_storage() for t, _, _ in parts]
        arr[i] = WpAdamWTensor(p.data_ptr(), None if ma is None else ma.data_ptr(), parts[0][0].data_ptr(),
                               parts[1][0].data_ptr(), parts[2][0].data_ptr() if eight else None,
                               parts[3][0].data_ptr() if eight else None, numel, _DT[p.dtype], 8 if eight else 32)
    _one_device("lora_adamw_plan", params[0])
    lib = _load()
    table = torch.empty(max(1, lib.lora_adamw_plan_size(arr, n)), dtype=torch.uint8, device=device)
    c = WpAdamWPlan()
    _check(lib.lora_adamw_plan_init(arr, n, table.data_ptr(), table.numel(), ctypes.byref(c), _stream(device)),
           "lora_adamw_plan")
    return AdamWPlan(c, table, kept, [p.numel() for p in params])


def lora_adamw_step(plan: AdamWPlan, grads: Sequence[Optional[torch.Tensor]], lr: float, beta1: float = 0.9,
                    beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01, step: int = 1,
                    grad_scale: float = 1.0, grad_scale_tensor: Optional[torch.Tensor] = None) -> None:
    """One AdamW step, in place, over the plan's tensors.  ``grads``: one per tensor, contiguous, all
    fp32 or all bf16; None leaves its tensor untouched.  ``grad_scale_tensor``: a device fp32 scalar
    that multiplies the gradients as well (a clip or loss scale).  A captured graph replays the ``lr``,
    ``step`` and other numbers that it was captured with."""
    if len(grads) != len(plan._numels):
        raise ValueError("lora_adamw_step: one gradient (or None) per tensor")
    given = [g for g in grads if g is not None]
    if not given:
        return
    dtype = given[0].dtype
    if dtype not in _DT:
        raise ValueError("lora_adamw_step: gradients must be fp32 or bf16")
    numels = plan._numels if len(given) == len(grads) else [n for g, n in zip(grads, plan._numels) if g is not None]
    if [g.numel() for g in given] != numels or {g.dtype for g in given} != {dtype} \
            or not all([g.is_contiguous() for g in given]):
        raise ValueError("lora_adamw_step: a gradient has another dtype, size or layout than its tensor's")
    if grad_scale_tensor is not None and (grad_scale_tensor.dtype != torch.float32 or grad_scale_tensor.numel() != 1):
        raise ValueError("grad_scale_tensor must be one float32 value")
    device = _one_device("lora_adamw_step", plan._table, grad_scale_tensor, *given)
    ptrs = plan._pack_ptrs(*[0 if g is None else g.data_ptr() for g in grads])
    args = _pack_adamw(lr, beta1, beta2, eps, weight_decay, grad_scale, step,
                       0 if grad_scale_tensor is None else grad_scale_tensor.data_ptr())
    st = _load().lora_adamw_step(plan._packed, ptrs, _DT[dtype], args, _raw_stream(device))
    if st:
        _check(st, "lora_adamw_step")


def lora_block8_decode(codes: torch.Tensor, absmax: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The fp32 values of 8-bit moments (int8 codes: first moments; uint8: second moments)."""
    if codes.dtype not in (torch.int8, torch.uint8) or not codes.is_contiguous() or not absmax.is_contiguous() \
            or absmax.dtype != torch.float32 or absmax.numel() != (codes.numel() + 255) // 256:
        raise ValueError("lora_block8_decode: contiguous int8 or uint8 codes and one fp32 scale per 256 of them")
    device = _one_device("lora_block8_decode", codes, absmax, out)
    if out is None:
        out = torch.empty(codes.shape, dtype=torch.float32, device=codes.device)
    elif out.dtype != torch.float32 or out.numel() != codes.numel() or not out.is_contiguous():
        raise ValueError("lora_block8_decode: out must be contiguous fp32 of the codes' size")
    _check(_load().lora_block8_decode(codes.data_ptr(), codes.dtype == torch.int8, absmax.data_ptr(), codes.numel(),
                                      out.data_ptr(), _raw_stream(device)), "lora_block8_decode")
    return out


def lora_device_status(reset: bool = True) -> int:
    """The device status word (0, or -7 after a bounded wait expired).  Synchronises."""
    torch.cuda.synchronize()
    return _load().lora_device_status(1 if reset else 0)


def lora_set_wait_limit(timeout_ns: int) -> None:
    """How long a bounded device wait spins before its kernel gives up (default 2 s)."""
    _check(_load().lora_set_wait_limit(int(timeout_ns)), "lora_set_wait_limit")


def lora_nf4_codebook() -> list:
    buf = (ctypes.c_float * 16)()
    _load().lora_nf4_codebook(buf)
    return list(buf)


def lora_status_string(status: int) -> str:
    return _load().lora_status_string(status).decode()
