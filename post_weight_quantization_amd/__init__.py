"""Python binding of libgptq_mi355x (ctypes): argument marshalling only.

Every step of the method runs in the library's HIP kernels; PyTorch supplies device memory
and the current stream.  There is no fallback: without the built library or a GPU the calls
raise.  Names follow the C ABI in ``include/gptq.h``:

* :func:`gptq_fold` -- H -> U, hdiag, dead, report
* :func:`gptq_ladder` -- W, dead -> lost, tab
* :func:`gptq_sweep` -- W, U, hdiag, dead, tab, lost -> nib, rung, scale, E
* :func:`gptq_linear` -- X, codes, scale -> act(X W^T + bias) + residual
* :func:`gptq_gated` -- X, two members' codes and scales -> act(X Wg^T + bg) * (X Wu^T + bu)
* :func:`gptq_linear_backward`, :func:`gptq_gated_backward` -- the gradients of X
* :func:`gptq_rotary` -- rotary positions
* :func:`gptq_cache_write`, :func:`gptq_cache_read`, :func:`gptq_cache_attention` -- a 4-bit attention cache
* :func:`gptq_cache_score`, :func:`gptq_cache_evict` -- its tokens' attention added up, and eviction by it
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import NamedTuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgptq_mi355x.so")

GPTQ_OK, GPTQ_EINVAL, GPTQ_EWORKSPACE, GPTQ_EHIP, GPTQ_DEGENERATE, GPTQ_ECHECK, GPTQ_ETOOBIG = 0, 1, 2, 3, 4, 5, 6
GPTQ_PACKED_UPPER = -1  # ldh of a Hessian stored as its packed upper triangle

_lib = None


class GptqError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


class FoldReport(ctypes.Structure):
    _fields_ = [("lambda_used", ctypes.c_double), ("base", ctypes.c_double),
                ("damp", ctypes.c_double), ("attempts", ctypes.c_int32),
                ("n_dead", ctypes.c_int32), ("degenerate", ctypes.c_int32),
                ("precision", ctypes.c_int32), ("min_pivot", ctypes.c_double)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


# Arithmetic of the fold (include/gptq.h, GPTQ_FOLD_*).
FOLD_PRECISION = {"auto": 0, "f32": 1, "f64": 2}
# Codecs of a round's members (GPTQ_CODEC_*).
CODEC = {"q4tp": 0, "q2tp": 1}
# Element types and activations of the operators on quantized operands (GPTQ_F32.., GPTQ_ACT_*).
DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
EXACT_WEIGHTS = 16  # GPTQ_EXACT_WEIGHTS
ACT = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
ROTARY = {"half": 0, "interleaved": 1}  # GPTQ_ROTARY_*


class RoundMember(ctypes.Structure):
    """gptq_member of include/gptq.h."""
    _fields_ = [("W", ctypes.c_void_p), ("rows", ctypes.c_int64), ("codec", ctypes.c_int32),
                ("pad", ctypes.c_int32), ("lost", ctypes.c_void_p), ("tab", ctypes.c_void_p),
                ("codes", ctypes.c_void_p), ("rung", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


class RoundGroup(ctypes.Structure):
    """gptq_group of include/gptq.h."""
    _fields_ = [("H", ctypes.c_void_p), ("n", ctypes.c_int64), ("ldh", ctypes.c_int64),
                ("lam", ctypes.c_double), ("precision", ctypes.c_int32),
                ("members", ctypes.c_int32), ("member", ctypes.POINTER(RoundMember)),
                ("hdiag", ctypes.c_void_p), ("dead", ctypes.c_void_p), ("report", FoldReport),
                ("status", ctypes.c_int32), ("pad", ctypes.c_int32)]


class KVCache(NamedTuple):
    """The 4-bit attention cache's planes (include/gptq.h, gptq_cache): k, v u8 [pages, heads, page,
    dim / 2], k_scale, v_scale bf16 [pages, heads, page, dim / 32].  The cache calls take any such
    four tensors."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


# gptq_cache and gptq_batch of include/gptq.h, in their fields' order (no padding between them).
_CACHE = struct.Struct("=QQQQqiiii").pack
_BATCH = struct.Struct("=QQQiiq").pack
_WEIGHTS = struct.Struct("=QQQ").pack  # gptq_weights
_ROTATED = struct.Struct("=QqqQqqii").pack  # gptq_rotated


def load():
    """Load the in-tree library (built by ``build.build()``); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m post_weight_quantization_amd.build` (hipcc, gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    P, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    lib.gptq_fold_workspace_size.argtypes = [i64]
    lib.gptq_fold_workspace_size.restype = sz
    lib.gptq_fold_workspace_size_ex.argtypes = [i64, ctypes.c_int]
    lib.gptq_fold_workspace_size_ex.restype = sz
    lib.gptq_fold.argtypes = [P, i64, i64, ctypes.c_double, P, P, P, P, sz, P,
                              ctypes.POINTER(FoldReport)]
    lib.gptq_fold.restype = ctypes.c_int
    lib.gptq_fold_ex.argtypes = [P, i64, i64, ctypes.c_double, ctypes.c_int, P, P, P, P, sz, P,
                                 ctypes.POINTER(FoldReport)]
    lib.gptq_fold_ex.restype = ctypes.c_int
    lib.gptq_ladder.argtypes = [P, P, i64, i64, P, P, P]
    lib.gptq_ladder.restype = ctypes.c_int
    lib.gptq_sweep_workspace_size.argtypes = [i64, i64]
    lib.gptq_sweep_workspace_size.restype = sz
    lib.gptq_sweep.argtypes = [P, P, P, P, P, P, i64, i64, P, P, P, P, P, sz, P]
    lib.gptq_sweep.restype = ctypes.c_int
    lib.gptq_sweep_inplace_workspace_size.argtypes = [i64, i64]
    lib.gptq_sweep_inplace_workspace_size.restype = sz
    lib.gptq_sweep_inplace.argtypes = [P, P, P, P, P, P, i64, i64, P, P, P, P, P, sz, P]
    lib.gptq_sweep_inplace.restype = ctypes.c_int
    lib.gptq_sweep_inplace_noalloc.argtypes = [P, P, P, P, P, P, i64, i64, P, P, P, P, P]
    lib.gptq_sweep_inplace_noalloc.restype = ctypes.c_int
    lib.gptq_gram_add.argtypes = [P, i64, i64, P, i64, i64, P]
    lib.gptq_gram_add.restype = ctypes.c_int
    lib.gptq_debias_workspace_size.argtypes = [i64, i64]
    lib.gptq_debias_workspace_size.restype = sz
    lib.gptq_debias.argtypes = [P, P, i64, P, P, P, P, P, P, P, i64, i64, P, sz, P]
    lib.gptq_debias.restype = ctypes.c_int
    lib.gptq_act_order_perm.argtypes = [P, i64, i64, P, P, P]
    lib.gptq_act_order_perm.restype = ctypes.c_int
    lib.gptq_permute_hessian.argtypes = [P, i64, i64, P, P, P]
    lib.gptq_permute_hessian.restype = ctypes.c_int
    lib.gptq_sweep_act_order_workspace_size.argtypes = [i64, i64]
    lib.gptq_sweep_act_order_workspace_size.restype = sz
    lib.gptq_sweep_act_order.argtypes = [P, P, P, P, P, P, i64, i64, P, P, P, P, P, sz, P]
    lib.gptq_sweep_act_order.restype = ctypes.c_int
    lib.gptq_sweep_act_order_q2.argtypes = [P, P, P, P, P, P, i64, i64, P, P, P, P, P, sz, P]
    lib.gptq_sweep_act_order_q2.restype = ctypes.c_int
    lib.gptq_debias_q2.argtypes = [P, P, i64, P, P, P, P, P, P, P, i64, i64, P, sz, P]
    lib.gptq_debias_q2.restype = ctypes.c_int
    lib.gptq_ladder_q2.argtypes = [P, P, i64, i64, P, P, P]
    lib.gptq_ladder_q2.restype = ctypes.c_int
    lib.gptq_sweep_q2.argtypes = [P, P, P, P, P, i64, i64, P, P, P, P, P, sz, P]
    lib.gptq_sweep_q2.restype = ctypes.c_int
    lib.gptq_round_slot_size.argtypes = [ctypes.POINTER(RoundGroup), ctypes.c_int32]
    lib.gptq_round_slot_size.restype = sz
    lib.gptq_round_plan.argtypes = [ctypes.POINTER(RoundGroup), ctypes.c_int32, sz, ctypes.c_int32,
                                    ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
    lib.gptq_round_plan.restype = ctypes.c_int
    lib.gptq_round.argtypes = [ctypes.POINTER(RoundGroup), ctypes.c_int32, P, sz, ctypes.c_int32, P]
    lib.gptq_round.restype = ctypes.c_int
    lib.gptq_linear_workspace_size.argtypes = [ctypes.c_int, i64, i64, i64]
    lib.gptq_linear_workspace_size.restype = sz
    lib.gptq_linear.argtypes = [P, i64, ctypes.c_int, i64, ctypes.c_int, P, P, i64, i64, P, ctypes.c_int, P, i64, P,
                                i64, P, sz, P]
    lib.gptq_linear.restype = ctypes.c_int
    cp = bp = ctypes.c_char_p  # the structs as bytes
    lib.gptq_cache_write.argtypes = [cp, bp, P, P, i64, i64, ctypes.c_int, P]
    lib.gptq_cache_write.restype = ctypes.c_int
    lib.gptq_cache_read.argtypes = [cp, bp, P, P, i64, i64, ctypes.c_int, P]
    lib.gptq_cache_read.restype = ctypes.c_int
    lib.gptq_cache_attention_workspace_size.argtypes = [cp, bp, ctypes.c_int32, ctypes.c_int]
    lib.gptq_cache_attention_workspace_size.restype = sz
    lib.gptq_cache_attention.argtypes = [cp, bp, P, i64, i64, ctypes.c_int32, ctypes.c_int, ctypes.c_float,
                                         ctypes.c_int32, ctypes.c_int32, P, i64, i64, P, P, sz, P]
    lib.gptq_cache_attention.restype = ctypes.c_int
    i32, ci, cf = ctypes.c_int32, ctypes.c_int, ctypes.c_float
    for name in ("gptq_linear_backward", "gptq_gated", "gptq_gated_backward"):
        size = getattr(lib, name + "_workspace_size")
        size.argtypes = [ci, i64, i64, i64]
        size.restype = sz
    lib.gptq_linear_backward.argtypes = [P, i64, ci, i64, ci, P, P, i64, i64, P, i64, P, sz, P]
    lib.gptq_linear_backward.restype = ci
    lib.gptq_gated.argtypes = [P, i64, ci, i64, ci, cp, cp, i64, i64, ci, P, i64, P, sz, P]
    lib.gptq_gated.restype = ci
    lib.gptq_gated_backward.argtypes = [P, i64] + lib.gptq_gated.argtypes
    lib.gptq_gated_backward.restype = ci
    lib.gptq_rotary.argtypes = [cp, i32, ci, i64, i32, i32, ci, P, P, cf, ci, P]
    lib.gptq_rotary.restype = ci
    lib.gptq_cache_score.argtypes = [cp, bp, P, i64, i64, i32, ci, cf, i32, i32, P, P, P, P]
    lib.gptq_cache_score.restype = ci
    lib.gptq_cache_evict.argtypes = [cp, bp, P, i32, i32, i32, P, i32, P, P, P]
    lib.gptq_cache_evict.restype = ci
    lib.gptq_status_string.argtypes = [ctypes.c_int]
    lib.gptq_status_string.restype = ctypes.c_char_p
    lib.gptq_profile_enable.argtypes = [ctypes.c_uint]
    lib.gptq_profile_enable.restype = None
    lib.gptq_profile_collect.argtypes = [P, P, P, P, ctypes.c_int]
    lib.gptq_profile_collect.restype = ctypes.c_int
    lib.gptq_profile_family_count.restype = ctypes.c_int
    lib.gptq_profile_family_name.argtypes = [ctypes.c_int]
    lib.gptq_profile_family_name.restype = ctypes.c_char_p
    lib.gptq_check_mode.argtypes = [ctypes.c_int]
    lib.gptq_check_mode.restype = None
    lib.gptq_check_message.restype = ctypes.c_char_p
    lib.gptq_check_selftest.argtypes = [ctypes.c_int]
    lib.gptq_check_selftest.restype = ctypes.c_int
    lib.gptq_check_tile_order.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    lib.gptq_check_tile_order.restype = ctypes.c_int
    lib.gptq_check_cache_row.argtypes = [i64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, ctypes.c_int32, i64,
                                         ctypes.c_int32]
    lib.gptq_check_cache_row.restype = i64
    lib.gptq_check_linear_plan.argtypes = [ctypes.c_int, i64, i64, i64, ctypes.POINTER(i64)]
    lib.gptq_check_linear_plan.restype = ctypes.c_int
    lib.gptq_check_backward_plan.argtypes = lib.gptq_check_linear_plan.argtypes
    lib.gptq_check_backward_plan.restype = ctypes.c_int
    lib.gptq_check_gated_plan.argtypes = [ci, i64, i64, i64, ci, ctypes.POINTER(i64)]
    lib.gptq_check_gated_plan.restype = ctypes.c_int
    lib.gptq_check_attention_blocks.argtypes = [ctypes.c_int32] * 3 + [i64] + [ctypes.c_int32] * 5
    lib.gptq_check_attention_blocks.restype = ctypes.c_int
    _lib = lib
    return lib


def require_native():
    """Raise unless the HIP library loads and a GPU is visible."""
    load()
    if not torch.cuda.is_available():
        raise RuntimeError("libgptq_mi355x needs a visible MI355X GPU")


def status_string(status: int) -> str:
    try:
        return load().gptq_status_string(int(status)).decode()
    except Exception:
        return "unknown"


def _dev(t: torch.Tensor, dtype, name, shape=None, align=1, device=None):
    """A contiguous device tensor's pointer, after checking its dtype, shape, device and the
    alignment (bytes) of its first element."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's tensors on {device}")
    if align > 1 and t.data_ptr() % align:
        raise ValueError(f"{name} must be {align}-byte aligned")
    return ctypes.c_void_p(t.data_ptr())


def _dev_rows(t: torch.Tensor, dtype, name):
    """A 2-D device tensor whose rows may be padded: unit column stride, row stride >= width
    (the row stride is passed as the leading dimension)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if t.dim() != 2 or (t.shape[0] > 1 and t.stride(1) != 1) or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return ctypes.c_void_p(t.data_ptr())


def _hessian(H: torch.Tensor, device=None):
    """(pointer, n, ldh) of a Hessian: a 2-D [n, n] tensor (rows may be padded) is passed as
    dense rows; a 1-D tensor of n (n + 1) / 2 floats as the packed upper triangle, row by row
    (ldh = GPTQ_PACKED_UPPER)."""
    if isinstance(H, torch.Tensor) and H.dim() == 1:
        P = H.numel()
        n = (math.isqrt(8 * P + 1) - 1) // 2
        if n < 1 or n * (n + 1) // 2 != P:
            raise ValueError("a packed H must hold n (n + 1) / 2 floats")
        return _dev(H, torch.float32, "H", device=device), n, GPTQ_PACKED_UPPER
    if not isinstance(H, torch.Tensor) or H.dim() != 2 or H.shape[0] != H.shape[1]:
        raise ValueError("H must be [n, n], or its packed upper triangle (1-D)")
    if device is not None and H.device != device:
        raise ValueError(f"H is on {H.device}, the call's tensors on {device}")
    return _dev_rows(H, torch.float32, "H"), H.shape[0], H.stride(0)


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream, device):
    """The stream a call is enqueued on, as a context for the tensors it allocates: PyTorch's
    caching allocator then reuses their memory only in that stream's order, after the call's
    kernels, never while they may still run."""
    s = torch.cuda.current_stream(device) if stream is None else stream
    return torch.cuda.stream(s)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _guards:
    """The device and stream guards of a call made elsewhere than where it runs."""
    __slots__ = ("all",)

    def __init__(self, *guards):
        self.all = [g for g in guards if g is not None]

    def __enter__(self):
        for g in self.all:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.all):
            g.__exit__(*exc)
        return False


_HERE = _guards()


def _at(stream, index):
    """(guard, stream handle) of a call on device ``index``, whatever is current: what is allocated under
    the guard belongs to that device and stream.  The usual case, both current, costs little."""
    if stream is None:
        handle = _raw_stream(index) if _raw_stream else torch.cuda.current_stream(index).cuda_stream
        return (_HERE if index == torch.cuda.current_device() else _guards(torch.cuda.device(index))), handle
    if stream.device.index != index:
        raise ValueError(f"the stream is on {stream.device}, the call's tensors on cuda:{index}")
    return (_guards(torch.cuda.device(index) if index != torch.cuda.current_device() else None,
                    torch.cuda.stream(stream)), stream.cuda_stream)


def _ptr(t, dtype, name, shape, index, align=1):
    """The address of a contiguous tensor on device ``index``: _dev's checks in their shortest form, and its
    messages."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != index \
            or not t.is_contiguous():
        _dev(t, dtype, name, shape, align, torch.device("cuda", index))
    p = t.data_ptr()
    if p & (align - 1):
        raise ValueError(f"{name} must be {align}-byte aligned")
    return p


def _workspace(workspace, need, device, name="workspace"):
    if workspace is None:
        return torch.empty(max(int(need), 1), dtype=torch.uint8, device=device)
    _dev(workspace, torch.uint8, name, align=256, device=device)
    if workspace.numel() < need:
        raise ValueError(f"{name} has {workspace.numel()} bytes, the call needs {need}")
    return workspace


def fold_workspace_size(n: int, precision: str = "auto") -> int:
    return int(load().gptq_fold_workspace_size_ex(int(n), FOLD_PRECISION[precision]))


def sweep_workspace_size(rows: int, n: int) -> int:
    return int(load().gptq_sweep_workspace_size(int(rows), int(n)))


def gptq_fold(H: torch.Tensor, lam: float, workspace: torch.Tensor | None = None, stream=None,
              out=None, check=True, precision: str = "auto"):
    """Fold H (f32 [n, n], upper triangle read, rows may be padded; or its packed upper
    triangle, 1-D).  ``precision`` is "auto" (f32, repeated in f64 where a pivot is at or below
    1e-2), "f32" or "f64".  Returns (U, hdiag, dead, report dict)."""
    lib = load()
    dev = H.device
    h_ptr, n, ldh = _hessian(H)
    prec = FOLD_PRECISION[precision]
    need = int(lib.gptq_fold_workspace_size_ex(n, prec))
    with _on(stream, dev):
        if out is None:
            U = torch.empty(n, n, dtype=torch.float32, device=dev)
            hdiag = torch.empty(n, dtype=torch.float32, device=dev)
            dead = torch.empty(n, dtype=torch.uint8, device=dev)
        else:
            U, hdiag, dead = out
        workspace = _workspace(workspace, need, dev)
    rep = FoldReport()
    st = lib.gptq_fold_ex(h_ptr, n, ldh, float(lam), prec,
                          _dev(U, torch.float32, "U", (n, n), device=dev),
                          _dev(hdiag, torch.float32, "hdiag", (n,), device=dev),
                          _dev(dead, torch.uint8, "dead", (n,), device=dev),
                          ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                          _stream(stream), ctypes.byref(rep))
    if check and st not in (GPTQ_OK, GPTQ_DEGENERATE):
        raise GptqError(st, "gptq_fold")
    r = rep.as_dict()
    r["status"] = st
    return U, hdiag, dead, r


def gptq_ladder(W: torch.Tensor, dead: torch.Tensor, stream=None, out=None):
    """Per-row (lo, step) and the 32 rung scales of the dead-zeroed W."""
    lib = load()
    rows, n = W.shape
    dev = W.device
    with _on(stream, dev):
        if out is None:
            lost = torch.empty(rows, 2, dtype=torch.float32, device=dev)
            tab = torch.empty(rows, 32, dtype=torch.float32, device=dev)
        else:
            lost, tab = out
    st = lib.gptq_ladder(_dev(W, torch.float32, "W", align=16), _dev(dead, torch.uint8, "dead", (n,), device=dev),
                         rows, n, _dev(lost, torch.float32, "lost", (rows, 2), device=dev),
                         _dev(tab, torch.float32, "tab", (rows, 32), device=dev), _stream(stream))
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_ladder")
    return lost, tab


def gptq_sweep(W, U, hdiag, dead, tab, lost, want_E=False, workspace=None, stream=None,
               out=None):
    """The q4tp sweep.  Returns (nib [rows, n/2] u8, rung [rows, n/32] u8,
    scale [rows, n/32] f32, E [rows, n] f32 or None)."""
    lib = load()
    rows, n = W.shape
    dev = W.device
    need = int(lib.gptq_sweep_workspace_size(rows, n))
    with _on(stream, dev):
        if out is None:
            nib = torch.empty(rows, n // 2, dtype=torch.uint8, device=dev)
            rung = torch.empty(rows, n // 32, dtype=torch.uint8, device=dev)
            scale = torch.empty(rows, n // 32, dtype=torch.float32, device=dev)
            E = torch.empty(rows, n, dtype=torch.float32, device=dev) if want_E else None
        else:
            nib, rung, scale, E = out
        workspace = _workspace(workspace, need, dev)
    st = lib.gptq_sweep(_dev(W, torch.float32, "W", align=16),
                        _dev(U, torch.float32, "U", (n, n), 16, dev),
                        _dev(hdiag, torch.float32, "hdiag", (n,), device=dev),
                        _dev(dead, torch.uint8, "dead", (n,), device=dev),
                        _dev(tab, torch.float32, "tab", (rows, 32), 16, dev),
                        _dev(lost, torch.float32, "lost", (rows, 2), 8, dev),
                        rows, n, _dev(nib, torch.uint8, "nib", (rows, n // 2), 16, dev),
                        _dev(rung, torch.uint8, "rung", (rows, n // 32), device=dev),
                        _dev(scale, torch.float32, "scale", (rows, n // 32), device=dev),
                        None if E is None else _dev(E, torch.float32, "E", (rows, n), 16, dev),
                        ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                        _stream(stream))
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_sweep")
    return nib, rung, scale, E


def gptq_sweep_inplace(W, U, hdiag, dead, tab, lost, want_E=False, workspace=None, stream=None,
                       out=None):
    """The q4tp sweep with W as its own working copy (W is overwritten).  Returns (nib, rung,
    scale, E or None), the same as :func:`gptq_sweep` on the original W."""
    lib = load()
    rows, n = W.shape
    dev = W.device
    with _on(stream, dev):
        if out is None:
            nib = torch.empty(rows, n // 2, dtype=torch.uint8, device=dev)
            rung = torch.empty(rows, n // 32, dtype=torch.uint8, device=dev)
            scale = torch.empty(rows, n // 32, dtype=torch.float32, device=dev)
            E = torch.empty(rows, n, dtype=torch.float32, device=dev) if want_E else None
        else:
            nib, rung, scale, E = out
        need = 0 if E is not None else int(lib.gptq_sweep_inplace_workspace_size(rows, n))
        if need:
            workspace = _workspace(workspace, need, dev)
    ws_ptr = ctypes.c_void_p(workspace.data_ptr()) if (need and workspace is not None) else None
    st = lib.gptq_sweep_inplace(_dev(W, torch.float32, "W", align=16),
                                _dev(U, torch.float32, "U", (n, n), 16, dev),
                                _dev(hdiag, torch.float32, "hdiag", (n,), device=dev),
                                _dev(dead, torch.uint8, "dead", (n,), device=dev),
                                _dev(tab, torch.float32, "tab", (rows, 32), 16, dev),
                                _dev(lost, torch.float32, "lost", (rows, 2), 8, dev),
                                rows, n, _dev(nib, torch.uint8, "nib", (rows, n // 2), device=dev),
                                _dev(rung, torch.uint8, "rung", (rows, n // 32), device=dev),
                                _dev(scale, torch.float32, "scale", (rows, n // 32), device=dev),
                                None if E is None else _dev(E, torch.float32, "E", (rows, n), 16, dev),
                                ws_ptr, workspace.numel() if ws_ptr is not None else 0,
                                _stream(stream))
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_sweep_inplace")
    return nib, rung, scale, E


def gptq_gram_add(H: torch.Tensor, X: torch.Tensor, stream=None):
    """H (f32 [n, n], device; or its packed upper triangle, 1-D) += X^T X on its upper
    triangle, X f32 [t, n] (tokens x channels).  Returns H."""
    lib = load()
    h_ptr, n, ldh = _hessian(H)
    if X.dim() != 2 or X.shape[1] != n:
        raise ValueError("X must be [t, n] with n = H.shape[0]")
    if X.device != H.device:
        raise ValueError("X and H must be on one device")
    st = lib.gptq_gram_add(h_ptr, n, ldh,
                           _dev_rows(X, torch.float32, "X"), X.shape[0], X.stride(0), _stream(stream))
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_gram_add")
    return H


def debias_workspace_size(rows: int, n: int) -> int:
    return int(load().gptq_debias_workspace_size(int(rows), int(n)))


def gptq_debias(W, H, dead, nib, rung, lost, scale, want_tab=True, want_slope=True,
                workspace=None, stream=None):
    """Output debias in place on (lost, scale).  Returns (lost, tab or None, scale,
    slope f64 [rows] or None)."""
    lib = load()
    rows, n = W.shape
    dev = W.device
    h_ptr, hn, ldh = _hessian(H, dev)
    if hn != n:
        raise ValueError(f"H has {hn} channels, W {n}")
    need = int(lib.gptq_debias_workspace_size(rows, n))
    with _on(stream, dev):
        tab = torch.empty(rows, 32, dtype=torch.float32, device=dev) if want_tab else None
        slope = torch.empty(rows, dtype=torch.float64, device=dev) if want_slope else None
        workspace = _workspace(workspace, need, dev)
    st = lib.gptq_debias(_dev(W, torch.float32, "W", align=16), h_ptr,
                         ldh, _dev(dead, torch.uint8, "dead", (n,), device=dev),
                         _dev(nib, torch.uint8, "nib", (rows, n // 2), 16, dev),
                         _dev(rung, torch.uint8, "rung", (rows, n // 32), device=dev),
                         _dev(lost, torch.float32, "lost", (rows, 2), 8, dev),
                         None if tab is None else _dev(tab, torch.float32, "tab", (rows, 32), 16, dev),
                         _dev(scale, torch.float32, "scale", (rows, n // 32), device=dev),
                         None if slope is None else _dev(slope, torch.float64, "slope", (rows,), device=dev),
                         rows, n, ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                         _stream(stream))
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_debias")
    return lost, tab, scale, slope


def gptq_debias_q2(W, H, dead, plane, rung, lost, scale, want_tab=True, want_slope=True,
                   workspace=None, stream=None):
    """Output debias of 2-bit codes in place on (lost, scale).  Returns (lost, tab or None,
    scale, slope f64 [rows] or None)."""
    lib = load()
    rows, n = W.shape
    dev = W.device
    h_ptr, hn, ldh = _hessian(H, dev)
    if hn != n:
        raise ValueError(f"H has {hn} channels, W {n}")
    need = int(lib.gptq_debias_workspace_size(rows, n))
    with _on(stream, dev):
        tab = torch.empty(rows, 32, dtype=torch.float32, device=dev) if want_tab else None
        slope = torch.empty(rows, dtype=torch.float64, device=dev) if want_slope else None
        workspace = _workspace(workspace, need, dev)
    st = lib.gptq_debias_q2(_dev(W, torch.float32, "W", align=16), h_ptr,
                            ldh, _dev(dead, torch.uint8, "dead", (n,), device=dev),
                            _dev(plane, torch.uint8, "plane", (rows, n // 4), device=dev),
                            _dev(rung, torch.uint8, "rung", (rows, n // 32), device=dev),
                            _dev(lost, torch.float32, "lost", (rows, 2), 8, dev),
                            None if tab is None else _dev(tab, torch.float32, "tab", (rows, 32), 16, dev),
                            _dev(scale, torch.float32, "scale", (rows, n // 32), device=dev),
                            None if slope is None else _dev(slope, torch.float64, "slope", (rows,), device=dev),
                            rows, n, ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                            _stream(stream))
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_debias_q2")
    return lost, tab, scale, slope


def gptq_sweep_act_order_q2(W, U, dead, hdiag, perm, tab, want_E=False, workspace=None,
                            stream=None):
    """Act-order q2tp sweep.  ``U`` and ``hdiag`` come from the fold of H[perm][perm] (hdiag
    in elimination order); ``dead`` in original order.  Returns (plane [rows, n/4], rung,
    scale, E or None); E in elimination order."""
    lib = load()
    rows, n = W.shape
    dev = W.device
    need = int(lib.gptq_sweep_act_order_workspace_size(rows, n))
    with _on(stream, dev):
        plane = torch.empty(rows, n // 4, dtype=torch.uint8, device=dev)
        rung = torch.empty(rows, n // 32, dtype=torch.uint8, device=dev)
        scale = torch.empty(rows, n // 32, dtype=torch.float32, device=dev)
        E = torch.empty(rows, n, dtype=torch.float32, device=dev) if want_E else None
        workspace = _workspace(workspace, need, dev)
    st = lib.gptq_sweep_act_order_q2(_dev(W, torch.float32, "W", align=16),
                                     _dev(U, torch.float32, "U", (n, n), 16, dev),
                                     _dev(dead, torch.uint8, "dead", (n,), device=dev),
                                     _dev(hdiag, torch.float32, "hdiag", (n,), device=dev),
                                     _dev(perm, torch.int32, "perm", (n,), device=dev),
                                     _dev(tab, torch.float32, "tab", (rows, 32), 16, dev),
                                     rows, n, _dev(plane, torch.uint8, "plane"),
                                     _dev(rung, torch.uint8, "rung"), _dev(scale, torch.float32, "scale"),
                                     None if E is None else _dev(E, torch.float32, "E"),
                                     ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                                     _stream(stream))
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_sweep_act_order_q2")
    return plane, rung, scale, E


def gptq_ladder_q2(W, dead, stream=None):
    """The q2tp ladder: (lost [rows, 2], tab [rows, 32]) with TAB[0] = 0."""
    lib = load()
    rows, n = W.shape
    dev = W.device
    with _on(stream, dev):
        lost = torch.empty(rows, 2, dtype=torch.float32, device=dev)
        tab = torch.empty(rows, 32, dtype=torch.float32, device=dev)
    st = lib.gptq_ladder_q2(_dev(W, torch.float32, "W", align=16),
                            _dev(dead, torch.uint8, "dead", (n,), device=dev), rows, n,
                            _dev(lost, torch.float32, "lost"), _dev(tab, torch.float32, "tab"),
                            _stream(stream))
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_ladder_q2")
    return lost, tab


def gptq_sweep_q2(W, U, hdiag, dead, tab, want_E=False, workspace=None, stream=None):
    """The q2tp sweep ("placed" rule).  Returns (plane [rows, n/4] u8, rung, scale, E or None)."""
    lib = load()
    rows, n = W.shape
    dev = W.device
    need = int(lib.gptq_sweep_workspace_size(rows, n))
    with _on(stream, dev):
        plane = torch.empty(rows, n // 4, dtype=torch.uint8, device=dev)
        rung = torch.empty(rows, n // 32, dtype=torch.uint8, device=dev)
        scale = torch.empty(rows, n // 32, dtype=torch.float32, device=dev)
        E = torch.empty(rows, n, dtype=torch.float32, device=dev) if want_E else None
        workspace = _workspace(workspace, need, dev)
    st = lib.gptq_sweep_q2(_dev(W, torch.float32, "W", align=16),
                           _dev(U, torch.float32, "U", (n, n), 16, dev),
                           _dev(hdiag, torch.float32, "hdiag", (n,), device=dev),
                           _dev(dead, torch.uint8, "dead", (n,), device=dev),
                           _dev(tab, torch.float32, "tab", (rows, 32), 16, dev), rows, n,
                           _dev(plane, torch.uint8, "plane"), _dev(rung, torch.uint8, "rung"),
                           _dev(scale, torch.float32, "scale"),
                           None if E is None else _dev(E, torch.float32, "E"),
                           ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                           _stream(stream))
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_sweep_q2")
    return plane, rung, scale, E


def sweep_act_order_workspace_size(rows: int, n: int) -> int:
    return int(load().gptq_sweep_act_order_workspace_size(int(rows), int(n)))


def gptq_act_order_perm(H, stream=None):
    """(perm i32 [n], dead u8 [n]) of act-order GPTQ from H's diagonal (H dense or packed)."""
    lib = load()
    dev = H.device
    h_ptr, n, ldh = _hessian(H)
    with _on(stream, dev):
        perm = torch.empty(n, dtype=torch.int32, device=dev)
        dead = torch.empty(n, dtype=torch.uint8, device=dev)
    st = lib.gptq_act_order_perm(h_ptr, n, ldh,
                                 _dev(perm, torch.int32, "perm"), _dev(dead, torch.uint8, "dead"),
                                 _stream(stream))
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_act_order_perm")
    return perm, dead


def gptq_permute_hessian(H, perm, stream=None):
    """H[perm][perm] (f32 [n, n], full symmetric) from H's upper triangle (H dense or
    packed)."""
    lib = load()
    dev = H.device
    h_ptr, n, ldh = _hessian(H)
    with _on(stream, dev):
        Hp = torch.empty(n, n, dtype=torch.float32, device=dev)
    st = lib.gptq_permute_hessian(h_ptr, n, ldh,
                                  _dev(perm, torch.int32, "perm", (n,), device=dev),
                                  _dev(Hp, torch.float32, "Hp"), _stream(stream))
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_permute_hessian")
    return Hp


def gptq_sweep_act_order(W, U, dead, perm, tab, lost, want_E=False, workspace=None, stream=None):
    """Act-order q4tp sweep.  Returns (nib, rung, scale, E or None); E in elimination order."""
    lib = load()
    rows, n = W.shape
    dev = W.device
    need = int(lib.gptq_sweep_act_order_workspace_size(rows, n))
    with _on(stream, dev):
        nib = torch.empty(rows, n // 2, dtype=torch.uint8, device=dev)
        rung = torch.empty(rows, n // 32, dtype=torch.uint8, device=dev)
        scale = torch.empty(rows, n // 32, dtype=torch.float32, device=dev)
        E = torch.empty(rows, n, dtype=torch.float32, device=dev) if want_E else None
        workspace = _workspace(workspace, need, dev)
    st = lib.gptq_sweep_act_order(_dev(W, torch.float32, "W", align=16),
                                  _dev(U, torch.float32, "U", (n, n), 16, dev),
                                  _dev(dead, torch.uint8, "dead", (n,), device=dev),
                                  _dev(perm, torch.int32, "perm", (n,), device=dev),
                                  _dev(tab, torch.float32, "tab", (rows, 32), 16, dev),
                                  _dev(lost, torch.float32, "lost", (rows, 2), 8, dev),
                                  rows, n, _dev(nib, torch.uint8, "nib"),
                                  _dev(rung, torch.uint8, "rung"), _dev(scale, torch.float32, "scale"),
                                  None if E is None else _dev(E, torch.float32, "E"),
                                  ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                                  _stream(stream))
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_sweep_act_order")
    return nib, rung, scale, E


def _no_history(what, *tensors):
    """Refuses tensors that a gradient is asked of: the operators on quantized operands leave no history (gradients are
    calls of their own, gptq_linear_backward, gptq_gated_backward and gptq_rotary's), and their outputs would drop it
    without a word."""
    for t in tensors:
        if getattr(t, "requires_grad", False) and torch.is_grad_enabled():
            raise ValueError(f"{what} has no gradient: call it under torch.no_grad() or on detached tensors")


def linear_workspace_size(t: int, rows: int, n: int, dtype=torch.bfloat16, exact: bool = False) -> int:
    return int(load().gptq_linear_workspace_size(DTYPE[dtype] | (EXACT_WEIGHTS if exact else 0), int(t), int(rows), int(n)))


def _matrix(t, dtype, name, rows, cols, index):
    """A 2-D tensor of a call whose rows may be padded: (pointer, row stride)."""
    if not isinstance(t, torch.Tensor) or t.shape != (rows, cols):
        raise ValueError(f"{name} must be a tensor of shape {(rows, cols)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the call's tensors on cuda:{index}")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    # A single row's stride is never used; torch gives it any value.
    return t.data_ptr(), ld if rows > 1 else cols


def gptq_linear(X, codes, scale, codec: str = "q4tp", bias=None, act: str = "none", residual=None, out=None,
                workspace=None, stream=None, exact: bool = False):
    """Y = act(X W^T + bias) + residual with W the weights that a sweep's codes stand for.  X [t, n]
    (rows may be padded) in f32, bf16 or f16, codes [rows, n/2] (q4tp) or [rows, n/4] (q2tp), scale
    [rows, n/32] f32, bias [rows] f32, residual [t, rows] like X; ``act`` a key of ACT.  ``out`` may
    be the residual itself and must not overlap another argument (X least of all: such a call raises
    GptqError).  With many tokens in bf16 or f16 the weights are rounded to that type; ``exact`` keeps them
    as they are at any number of tokens (include/gptq.h).  The gradient of X is :func:`gptq_linear_backward`'s; tensors that
    require one raise ValueError, unless gradients are switched off.  Returns Y [t, rows]."""
    lib = _lib or load()
    _no_history("gptq_linear", X, scale, bias, residual, out)
    if not isinstance(X, torch.Tensor) or not X.is_cuda or X.dim() != 2 or X.dtype not in DTYPE:
        raise ValueError("X must be a 2-D device tensor in float32, bfloat16 or float16")
    (t, n), kind, index = X.shape, X.dtype, X.get_device()
    if codec not in CODEC or act not in ACT:
        raise ValueError(f"codec must be one of {list(CODEC)}, act one of {list(ACT)}")
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise ValueError("codes must be [rows, n/2] (q4tp) or [rows, n/4] (q2tp)")
    rows, dt = codes.shape[0], DTYPE[kind] | (EXACT_WEIGHTS if exact else 0)
    xp, ldx = _matrix(X, kind, "X", t, n, index)
    if t == 1:  # any stride that its own alignment allows
        ldx = (n + 7) & ~7
    cp = _ptr(codes, torch.uint8, "codes", (rows, n // (2 if codec == "q4tp" else 4)), index, 16)
    sp = _ptr(scale, torch.float32, "scale", (rows, n // 32), index)
    bp = None if bias is None else _ptr(bias, torch.float32, "bias", (rows,), index)
    guard, s = _at(stream, index)
    with guard:
        if out is None:
            out = torch.empty(t, rows, dtype=kind, device=X.device)
        yp, ldy = _matrix(out, kind, "out", t, rows, index)
        rp, ldr = (None, 0) if residual is None else _matrix(residual, kind, "residual", t, rows, index)
        need = lib.gptq_linear_workspace_size(dt, t, rows, n)
        ws = _workspace(workspace, need, X.device) if need else None
        st = lib.gptq_linear(xp, ldx, dt, t, CODEC[codec], cp, sp, rows, n, bp, ACT[act], rp, ldr, yp, ldy,
                             None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), s)
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_linear")
    return out


def cache_alloc(pages: int, page: int, heads: int, dim: int, device="cuda") -> KVCache:
    """A cache of ``pages`` pages of ``page`` tokens, zeroed (``dim`` 64, 128 or 256)."""
    if pages < 1 or page < 16 or page % 16 or heads < 1 or dim not in (64, 128, 256):
        raise ValueError("a cache needs pages >= 1, page a multiple of 16, heads >= 1 and dim 64, 128 or 256")
    shape = (pages, heads, page)
    k, v = (torch.zeros(*shape, dim // 2, dtype=torch.uint8, device=device) for _ in range(2))
    ks, vs = (torch.zeros(*shape, dim // 32, dtype=torch.bfloat16, device=device) for _ in range(2))
    return KVCache(k, v, ks, vs)


def _cache(cache):
    """gptq_cache of four planes, as bytes: (struct, heads, dim, device index)."""
    k, v, ks, vs = cache
    if not isinstance(k, torch.Tensor) or k.dim() != 4 or not k.is_cuda:
        raise ValueError("the cache's k must be a device tensor [pages, heads, page, dim / 2]")
    shape, index = k.shape, k.get_device()
    pages, heads, page, half = shape
    scales = (pages, heads, page, half // 16)
    u8, bf = torch.uint8, torch.bfloat16
    return _CACHE(_ptr(k, u8, "k", shape, index, 16), _ptr(v, u8, "v", shape, index, 16),
                  _ptr(ks, bf, "k_scale", scales, index, 16), _ptr(vs, bf, "v_scale", scales, index, 16),
                  pages, page, heads, 2 * half, 0), heads, 2 * half, index


def _batch(table, length, start, rows, index):
    """gptq_batch of the sequences' arrays, as bytes."""
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [sequences, pages]")
    seqs, width = table.shape
    if start is None and rows != seqs:
        raise ValueError(f"without start the call has one row a sequence, {seqs}, not {rows}")
    i32 = torch.int32
    return _BATCH(_ptr(table, i32, "table", (seqs, width), index), _ptr(length, i32, "length", (seqs,), index),
                  0 if start is None else _ptr(start, i32, "start", (seqs + 1,), index), seqs, width, rows)


def _heads(t, name, dtype, rows, heads, dim, index):
    """(pointer, row stride, head stride) of a [rows, heads, dim] tensor with contiguous dim."""
    if not isinstance(t, torch.Tensor) or t.shape != (rows, heads, dim):
        raise ValueError(f"{name} must be [rows, heads, dim] = {(rows, heads, dim)}")
    if t.dtype != dtype or t.get_device() != index:
        raise ValueError(f"{name} must be {dtype} on cuda:{index}")
    ld, ldh, step = t.stride()
    if step != 1:
        raise ValueError(f"{name}'s channels must be contiguous")
    # Strides that torch leaves open (one row, one head) become those of a contiguous tensor.
    if heads == 1:
        ldh = dim
    return t.data_ptr(), ld if rows > 1 else heads * max(ldh, dim), ldh


def gptq_cache_write(cache, K, V, table, length, start=None, stream=None):
    """Quantise K, V [rows, heads, dim] (f32, bf16, f16; slices of one projection are fine) into the
    cache's pages.  ``length`` [sequences] counts the cached tokens, these rows included; ``start``
    [sequences + 1] are the sequences' first rows (None: one row a sequence); ``table``
    [sequences, pages] i32 (include/gptq.h, gptq_batch).  No gradient: tensors that require one raise ValueError.  Returns the
    cache."""
    lib = _lib or load()
    _no_history("gptq_cache_write", K, V)
    c, heads, dim, index = _cache(cache)
    if not isinstance(K, torch.Tensor) or K.dim() != 3 or K.dtype not in DTYPE:
        raise ValueError("K must be a [rows, heads, dim] tensor in float32, bfloat16 or float16")
    rows, kind = K.shape[0], K.dtype
    kp, ld, ldh = _heads(K, "K", kind, rows, heads, dim, index)
    vp, ld2, ldh2 = _heads(V, "V", kind, rows, heads, dim, index)
    if ld != ld2 or ldh != ldh2:
        raise ValueError("K and V must have the same strides")
    b = _batch(table, length, start, rows, index)
    guard, s = _at(stream, index)
    with guard:
        st = lib.gptq_cache_write(c, b, kp, vp, ld, ldh, DTYPE[kind], s)
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_cache_write")
    return cache


def gptq_cache_read(cache, table, length, start=None, rows=None, dtype=torch.bfloat16, out=None, stream=None):
    """The cached values of a call's rows (as in :func:`gptq_cache_write`), dense: (K, V) of [rows,
    heads, dim].  ``rows``: how many rows the call has (None: one a sequence)."""
    lib = _lib or load()
    c, heads, dim, index = _cache(cache)
    rows = table.shape[0] if rows is None else int(rows)
    b = _batch(table, length, start, rows, index)
    guard, s = _at(stream, index)
    with guard:
        if out is None:
            if dtype not in DTYPE:
                raise ValueError("dtype must be float32, bfloat16 or float16")
            K, V = torch.empty(2, rows, heads, dim, dtype=dtype, device=cache[0].device).unbind()
        else:
            K, V = out
        kp, ld, ldh = _heads(K, "K", K.dtype, rows, heads, dim, index)
        vp, ld2, ldh2 = _heads(V, "V", K.dtype, rows, heads, dim, index)
        if ld != ld2 or ldh != ldh2 or K.dtype not in DTYPE:
            raise ValueError("K and V must have the same strides, in float32, bfloat16 or float16")
        st = lib.gptq_cache_read(c, b, kp, vp, ld, ldh, DTYPE[K.dtype], s)
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_cache_read")
    return K, V


def gptq_cache_attention(cache, Q, table, length, start=None, scale=None, window: int = 0, sinks: int = 0, out=None,
                         want_lse=False, workspace=None, stream=None):
    """softmax(scale Q K^T) V over the cache, causal: Q [rows, query heads, dim], rows and sequences as
    in :func:`gptq_cache_write`, ``scale`` 1 / sqrt(dim) when None.  A row at position p sees
    positions k <= p, and with a window only k > p - window or k < sinks; one that sees nothing gives
    zeros.  ``out`` may be Q itself (with its strides) and must not overlap an argument otherwise.
    No gradient: tensors that require one raise ValueError.  Returns O like Q, or (O, lse f32 [rows, query heads]) with ``want_lse``."""
    lib = _lib or load()
    _no_history("gptq_cache_attention", Q, out)
    c, heads, dim, index = _cache(cache)
    if not isinstance(Q, torch.Tensor) or Q.dim() != 3 or Q.dtype not in DTYPE:
        raise ValueError("Q must be a [rows, query heads, dim] device tensor in float32, bfloat16 or float16")
    (rows, qh, _), kind = Q.shape, Q.dtype
    dt = DTYPE[kind]
    if max(abs(int(window)), abs(int(sinks))) >= 1 << 31:
        raise ValueError("window and sinks must be below 2^31")
    qp, ldq, ldqh = _heads(Q, "Q", kind, rows, qh, dim, index)
    b = _batch(table, length, start, rows, index)
    guard, s = _at(stream, index)
    with guard:
        if out is None:
            out = torch.empty(rows, qh, dim, dtype=kind, device=Q.device)
        op, ldo, ldoh = _heads(out, "out", kind, rows, qh, dim, index)
        lse = torch.empty(rows, qh, dtype=torch.float32, device=Q.device) if want_lse else None
        need = lib.gptq_cache_attention_workspace_size(c, b, qh, dt)
        ws = _workspace(workspace, need, Q.device) if need else None
        st = lib.gptq_cache_attention(c, b, qp, ldq, ldqh, qh, dt, dim ** -0.5 if scale is None else float(scale),
                                      int(window), int(sinks), op, ldo, ldoh, None if lse is None else lse.data_ptr(),
                                      None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), s)
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_cache_attention")
    return (out, lse) if want_lse else out


def _weights(pair, bias, name, codec, n, index):
    """gptq_weights of a (codes, scale) pair, as bytes, and its rows."""
    codes, scale = pair
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise ValueError(f"{name} must be (codes [rows, n/2] (q4tp) or [rows, n/4] (q2tp), scale [rows, n/32])")
    rows = codes.shape[0]
    return _WEIGHTS(_ptr(codes, torch.uint8, f"{name}'s codes", (rows, n // (2 if codec == "q4tp" else 4)), index, 16),
                    _ptr(scale, torch.float32, f"{name}'s scale", (rows, n // 32), index),
                    0 if bias is None else _ptr(bias, torch.float32, f"{name}_bias", (rows,), index)), rows


def _activations(X, name):
    """(t, columns, dtype, device index) of a 2-D tensor of activations."""
    if not isinstance(X, torch.Tensor) or not X.is_cuda or X.dim() != 2 or X.dtype not in DTYPE:
        raise ValueError(f"{name} must be a 2-D device tensor in float32, bfloat16 or float16")
    return (*X.shape, X.dtype, X.get_device())


def linear_backward_workspace_size(t: int, rows: int, n: int, dtype=torch.bfloat16, exact: bool = False) -> int:
    return int(load().gptq_linear_backward_workspace_size(DTYPE[dtype] | (EXACT_WEIGHTS if exact else 0), int(t), int(rows), int(n)))


def gptq_linear_backward(dY, codes, scale, codec: str = "q4tp", out=None, workspace=None, stream=None, exact: bool = False):
    """dX = dY W, the gradient of :func:`gptq_linear`'s X (through its activation, multiply dY by that one's slope
    first).  dY [t, rows] (rows may be padded) in f32, bf16 or f16, codes and scale as there; ``out`` must not
    overlap an argument; ``exact`` as there.  Returns dX [t, n]."""
    lib = _lib or load()
    _no_history("gptq_linear_backward", dY, scale, out)
    t, rows, kind, index = _activations(dY, "dY")
    if codec not in CODEC:
        raise ValueError(f"codec must be one of {list(CODEC)}")
    if not isinstance(scale, torch.Tensor) or scale.dim() != 2:
        raise ValueError("scale must be [rows, n/32]")
    n, dt = 32 * scale.shape[1], DTYPE[kind] | (EXACT_WEIGHTS if exact else 0)
    dp, ldd = _matrix(dY, kind, "dY", t, rows, index)
    cp = _ptr(codes, torch.uint8, "codes", (rows, n // (2 if codec == "q4tp" else 4)), index, 16)
    sp = _ptr(scale, torch.float32, "scale", (rows, n // 32), index)
    guard, s = _at(stream, index)
    with guard:
        if out is None:
            out = torch.empty(t, n, dtype=kind, device=dY.device)
        xp, ldx = _matrix(out, kind, "out", t, n, index)
        need = lib.gptq_linear_backward_workspace_size(dt, t, rows, n)
        ws = _workspace(workspace, need, dY.device) if need else None
        st = lib.gptq_linear_backward(dp, ldd, dt, t, CODEC[codec], cp, sp, rows, n, xp, ldx,
                                      None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), s)
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_linear_backward")
    return out


def gated_workspace_size(t: int, rows: int, n: int, dtype=torch.bfloat16, backward: bool = False, exact: bool = False) -> int:
    size = load().gptq_gated_backward_workspace_size if backward else load().gptq_gated_workspace_size
    return int(size(DTYPE[dtype] | (EXACT_WEIGHTS if exact else 0), int(t), int(rows), int(n)))


def gptq_gated(X, gate, up, codec: str = "q4tp", act: str = "silu", gate_bias=None, up_bias=None, out=None, workspace=None,
               stream=None, exact: bool = False):
    """act(X Wg^T + gate_bias) * (X Wu^T + up_bias), the gated half of a feed-forward block: ``gate`` and ``up`` are
    (codes, scale) pairs of [rows, n] matrices as :func:`gptq_linear` takes them, X [t, n], biases [rows] f32.
    With many tokens the weights are rounded, to 11 bits in bf16 and 22 in f16; ``exact`` keeps them as they are.
    ``out`` must not overlap an argument.  The gradient of X is :func:`gptq_gated_backward`'s; tensors that require
    one raise ValueError, unless gradients are switched off.  Returns Y [t, rows]."""
    lib = _lib or load()
    _no_history("gptq_gated", X, gate[1], up[1], gate_bias, up_bias, out)
    t, n, kind, index = _activations(X, "X")
    return _gated(lib.gptq_gated, lib.gptq_gated_workspace_size, None, X, gate, up, codec, act, gate_bias, up_bias, out,
                  workspace, stream, exact, t, n, kind, index)


def gptq_gated_backward(dY, X, gate, up, codec: str = "q4tp", act: str = "silu", gate_bias=None, up_bias=None, out=None,
                        workspace=None, stream=None, exact: bool = False):
    """The gradient of :func:`gptq_gated`'s X from that of its result: dY [t, rows] like X, the other arguments that
    call's.  Both sums are made again, so X is all that has to be kept.  Returns dX [t, n]."""
    lib = _lib or load()
    _no_history("gptq_gated_backward", dY, X, gate[1], up[1], gate_bias, up_bias, out)
    t, n, kind, index = _activations(X, "X")
    return _gated(lib.gptq_gated_backward, lib.gptq_gated_backward_workspace_size, dY, X, gate, up, codec, act, gate_bias,
                  up_bias, out, workspace, stream, exact, t, n, kind, index)


def _gated(call, size, dY, X, gate, up, codec, act, gate_bias, up_bias, out, workspace, stream, exact, t, n, kind, index):
    if codec not in CODEC or act not in ACT:
        raise ValueError(f"codec must be one of {list(CODEC)}, act one of {list(ACT)}")
    dt = DTYPE[kind] | (EXACT_WEIGHTS if exact else 0)
    xp, ldx = _matrix(X, kind, "X", t, n, index)
    if t == 1:  # any stride that its own alignment allows
        ldx = (n + 7) & ~7
    wg, rows = _weights(gate, gate_bias, "gate", codec, n, index)
    wu, r2 = _weights(up, up_bias, "up", codec, n, index)
    if rows != r2:
        raise ValueError(f"gate has {rows} rows, up {r2}")
    first = () if dY is None else _matrix(dY, kind, "dY", t, rows, index)
    guard, s = _at(stream, index)
    with guard:
        wide = rows if dY is None else n
        if out is None:
            out = torch.empty(t, wide, dtype=kind, device=X.device)
        yp, ldy = _matrix(out, kind, "out", t, wide, index)
        need = size(dt, t, rows, n)
        ws = _workspace(workspace, need, X.device) if need else None
        st = call(*first, xp, ldx, dt, t, CODEC[codec], wg, wu, rows, n, ACT[act], yp, ldy,
                  None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), s)
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_gated" if dY is None else "gptq_gated_backward")
    return out


def rotary_frequencies(part: int, base: float = 10000.0, scaling: str = "none", stretch: float = 1.0, trained: int = 4096,
                       slow: float = 1.0, fast: float = 32.0, device="cuda"):
    """(freq f64 [part / 2], factor) for :func:`gptq_rotary`: pair i turns by base^(-2 i / part) a position.  For
    contexts ``stretch`` times the ``trained`` length, ``scaling`` is one of

    * "linear": all angles divided by stretch;
    * "base": base times stretch^(part / (part - 2)), which leaves the fastest pair as it is and divides the
      slowest's angle by stretch;
    * "ramp": pairs that turn more than ``fast`` times over the trained length stay, those that turn less than
      ``slow`` times are divided by stretch, linear in the turns in between; factor is 0.1 log(stretch) + 1."""
    if part < 2 or part % 2 or not base > 0 or not stretch >= 1 or trained < 1 or not fast > slow:
        raise ValueError("part must be even, base positive, stretch at least 1, trained at least 1, fast above slow")
    half, factor = part // 2, 1.0
    if scaling == "base":
        if part < 4:
            raise ValueError("a base can be stretched for part >= 4")
        base = base * stretch ** (part / (part - 2))
    freq = base ** (-torch.arange(half, dtype=torch.float64) / half)
    if scaling == "linear":
        freq = freq / stretch
    elif scaling == "ramp":
        keep = ((trained * freq / (2.0 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
        freq = freq * keep + freq / stretch * (1.0 - keep)
        factor = 0.1 * math.log(stretch) + 1.0
    elif scaling not in ("none", "base"):
        raise ValueError("scaling must be one of none, linear, base, ramp")
    return freq.to(device), factor


def gptq_rotary(Q, position, freq, K=None, layout: str = "half", factor: float = 1.0, backward: bool = False, out=None,
                stream=None):
    """Rotary positions on Q [rows, heads, dim], and on K [rows, its heads, dim] in the same launch: pairs of the first
    2 len(freq) channels (``layout`` "half": i and i + len(freq); "interleaved": 2 i and 2 i + 1) are turned by
    position freq and multiplied by ``factor``, the other channels are copied.  position [rows] i32, freq f64 (see
    :func:`rotary_frequencies`).  ``backward``: the gradients of Q and K from those of the results.  ``out``: a
    tensor, or with K a pair; each may be its own input (with its strides) and must not overlap another argument.  No
    history, as :func:`gptq_gated`.  Returns the turned Q, or (Q, K)."""
    lib = _lib or load()
    two = K is not None
    yq, yk = (None, None) if out is None else tuple(out) if two else (out, None)
    _no_history("gptq_rotary", Q, K, freq, yq, yk)
    if not isinstance(Q, torch.Tensor) or Q.dim() != 3 or not Q.is_cuda or Q.dtype not in DTYPE:
        raise ValueError("Q must be a [rows, heads, dim] device tensor in float32, bfloat16 or float16")
    if two and (not isinstance(K, torch.Tensor) or K.dim() != 3):
        raise ValueError("K must be a [rows, heads, dim] tensor")
    if layout not in ROTARY:
        raise ValueError(f"layout must be one of {list(ROTARY)}")
    (rows, hq, dim), kind, index = Q.shape, Q.dtype, Q.get_device()
    if not isinstance(freq, torch.Tensor) or freq.dim() != 1:
        raise ValueError("freq must be a 1-D float64 tensor")
    pairs = freq.shape[0]
    pp = _ptr(position, torch.int32, "position", (rows,), index)
    fp = _ptr(freq, torch.float64, "freq", (pairs,), index)
    guard, s = _at(stream, index)
    with guard:
        if yq is None:
            yq = torch.empty(rows, hq, dim, dtype=kind, device=Q.device)
        packed = _ROTATED(*_heads(Q, "Q", kind, rows, hq, dim, index), *_heads(yq, "Q's out", kind, rows, hq, dim, index), hq, 0)
        if two:
            hk = K.shape[1]
            if yk is None:
                yk = torch.empty(rows, hk, dim, dtype=kind, device=Q.device)
            packed += _ROTATED(*_heads(K, "K", kind, rows, hk, dim, index), *_heads(yk, "K's out", kind, rows, hk, dim, index), hk, 0)
        st = lib.gptq_rotary(packed, 2 if two else 1, DTYPE[kind], rows, dim, 2 * pairs, ROTARY[layout], pp, fp, factor,
                             1 if backward else 0, s)
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_rotary")
    return (yq, yk) if two else yq


def score_alloc(cache) -> torch.Tensor:
    """Scores beside a cache's pages, zeroed: f32 [pages, heads, page]."""
    return torch.zeros(cache[0].shape[:3], dtype=torch.float32, device=cache[0].device)


def gptq_cache_score(cache, Q, lse, score, table, length, start=None, scale=None, window: int = 0, sinks: int = 0, out=None,
                     stream=None):
    """Add the softmax weights that a call of :func:`gptq_cache_attention` gave its cached tokens to their scores
    (f32 [pages, heads, page], :func:`score_alloc`): the arguments are that call's, ``lse`` is what it returned with
    ``want_lse``.  Tokens that the call's rows are count from 0.  ``out``: other planes for the sums (None: score
    itself).  Returns the planes written."""
    lib = _lib or load()
    _no_history("gptq_cache_score", Q, lse, score, out)
    c, heads, dim, index = _cache(cache)
    if not isinstance(Q, torch.Tensor) or Q.dim() != 3 or Q.dtype not in DTYPE:
        raise ValueError("Q must be a [rows, query heads, dim] device tensor in float32, bfloat16 or float16")
    (rows, qh, _), kind = Q.shape, Q.dtype
    if max(abs(int(window)), abs(int(sinks))) >= 1 << 31:
        raise ValueError("window and sinks must be below 2^31")
    out = score if out is None else out
    qp, ldq, ldqh = _heads(Q, "Q", kind, rows, qh, dim, index)
    lp = _ptr(lse, torch.float32, "lse", (rows, qh), index)
    planes = cache[0].shape[:3]
    sp = _ptr(score, torch.float32, "score", planes, index)
    op = sp if out is score else _ptr(out, torch.float32, "out", planes, index)
    b = _batch(table, length, start, rows, index)
    guard, s = _at(stream, index)
    with guard:
        st = lib.gptq_cache_score(c, b, qp, ldq, ldqh, qh, DTYPE[kind], dim ** -0.5 if scale is None else float(scale),
                                  int(window), int(sinks), lp, sp, op, s)
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_cache_score")
    return out


def gptq_cache_evict(cache, table, length, score, keep: int, sinks: int = 0, recent: int = 0, into=None, out=None, stream=None):
    """Cut sequences back to ``keep`` tokens: per kv head the first ``sinks``, the last ``recent`` and of the others
    those with the highest scores, moved together in their order with their scores, in place or to the pages of
    ``into`` [sequences, pages] i32 (none of the sequences' own).  ``out``: (length [sequences], index [sequences, heads,
    keep]) i32 tensors for the results.  Returns them: tokens left, and old positions of what is kept, ascending,
    then -1 (include/gptq.h)."""
    lib = _lib or load()
    _no_history("gptq_cache_evict", score)
    c, heads, _, index = _cache(cache)
    keep, sinks, recent = int(keep), int(sinks), int(recent)
    if max(abs(keep), abs(sinks), abs(recent)) >= 1 << 31:
        raise ValueError("keep, sinks and recent must be below 2^31")
    sp = _ptr(score, torch.float32, "score", cache[0].shape[:3], index, 16)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [sequences, pages]")
    seqs = table.shape[0]
    b = _batch(table, length, None, seqs, index)
    ip, width = None, 0
    if into is not None:
        if not isinstance(into, torch.Tensor) or into.dim() != 2 or into.shape[0] != seqs:
            raise ValueError("into must be [sequences, pages]")
        width = into.shape[1]
        ip = _ptr(into, torch.int32, "into", (seqs, width), index)
    if keep < 1:
        raise ValueError("keep must be at least 1")
    guard, s = _at(stream, index)
    with guard:
        if out is None:
            device = score.device
            left = torch.empty(seqs, dtype=torch.int32, device=device)
            kept = torch.empty(seqs, heads, keep, dtype=torch.int32, device=device)
            lp, kp = left.data_ptr(), kept.data_ptr()
        else:
            left, kept = out
            lp = _ptr(left, torch.int32, "length's out", (seqs,), index)
            kp = _ptr(kept, torch.int32, "index's out", (seqs, heads, keep), index)
        st = lib.gptq_cache_evict(c, b, sp, keep, sinks, recent, ip, width, lp, kp, s)
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_cache_evict")
    return left, kept


PROFILE_FAMILIES = ["fold_update", "fold_panel", "fold_diag", "fold_build", "fold_make_u",
                    "sweep_group", "sweep_trail", "ladder", "fold_next", "sweep_next", "gram", "debias",
                    "linear", "cache", "attention"]


def profile_enable(families=None):
    """Time the named kernel families (all when None; none for an empty list)."""
    if families is None:
        mask = (1 << len(PROFILE_FAMILIES)) - 1
    else:
        mask = 0
        for f in families:
            mask |= 1 << PROFILE_FAMILIES.index(f)
    load().gptq_profile_enable(mask)


def profile_collect():
    """{family: dict(ms, launches, flops, bytes)} for the launches since the last collect."""
    import numpy as np
    lib = load()
    nf = lib.gptq_profile_family_count()
    ms = np.zeros(nf)
    ln = np.zeros(nf, dtype=np.int64)
    fl = np.zeros(nf)
    by = np.zeros(nf)
    P = ctypes.c_void_p
    st = lib.gptq_profile_collect(P(ms.ctypes.data), P(ln.ctypes.data), P(fl.ctypes.data),
                                  P(by.ctypes.data), nf)
    if st != GPTQ_OK:
        raise GptqError(st, "gptq_profile_collect")
    return {lib.gptq_profile_family_name(f).decode(): dict(ms=float(ms[f]), launches=int(ln[f]),
                                                           flops=float(fl[f]), bytes=float(by[f]))
            for f in range(nf)}


class Round:
    """A batched round (include/gptq.h, gptq_round) with its outputs and workspace allocated
    once, so that run() can be repeated.  ``groups``: a sequence of dicts with "H" (f32 [n, n],
    rows may be padded, or its packed upper triangle, 1-D), "lam", optionally "precision"
    ("auto", "f32", "f64"), and "members": W [rows, n] tensors, or (W, codec) pairs with codec
    "q4tp" or "q2tp".  Without a workspace, the slots the library's plan would use (its largest
    gang, or its threads), within half of the free device memory, are allocated.  ``results``: per group a dict with hdiag, dead and, per member, (lost, tab,
    codes, rung, scale); run() adds the group's status and fold report."""

    def __init__(self, groups, max_concurrency: int = 0, workspace=None, stream=None):
        lib = load()
        if not groups:
            raise ValueError("a round needs at least one group")
        dev = groups[0]["H"].device
        G = len(groups)
        self.arr = (RoundGroup * G)()
        self.keep, self.results = [], []
        with _on(stream, dev):
            for i, g in enumerate(groups):
                h_ptr, n, ldh = _hessian(g["H"], dev)
                mem = list(g.get("members", ()))
                ms = (RoundMember * max(len(mem), 1))()
                outs = []
                for k, m in enumerate(mem):
                    W, codec = m if isinstance(m, tuple) else (m, "q4tp")
                    if W.dim() != 2 or W.shape[1] != n:
                        raise ValueError(f"group {i} member {k}: W must be [rows, {n}]")
                    rows = W.shape[0]
                    cb = n // 2 if codec == "q4tp" else n // 4
                    o = (torch.empty(rows, 2, dtype=torch.float32, device=dev),
                         torch.empty(rows, 32, dtype=torch.float32, device=dev),
                         torch.empty(rows, cb, dtype=torch.uint8, device=dev),
                         torch.empty(rows, n // 32, dtype=torch.uint8, device=dev),
                         torch.empty(rows, n // 32, dtype=torch.float32, device=dev))
                    ms[k] = RoundMember(_dev(W, torch.float32, "W", align=16, device=dev).value,
                                        rows, CODEC[codec], 0, *(t.data_ptr() for t in o))
                    outs.append(o)
                hdiag = torch.empty(n, dtype=torch.float32, device=dev)
                dead = torch.empty(n, dtype=torch.uint8, device=dev)
                self.arr[i] = RoundGroup(h_ptr.value, n, ldh, float(g["lam"]),
                                         FOLD_PRECISION[g.get("precision", "auto")], len(mem), ms,
                                         hdiag.data_ptr(), dead.data_ptr(), FoldReport(), 0, 0)
                self.keep.append((ms, g["H"], mem))
                self.results.append(dict(hdiag=hdiag, dead=dead, members=outs))
            self.slot_bytes = int(lib.gptq_round_slot_size(self.arr, G))
            if self.slot_bytes == 0:
                raise ValueError("a group of the round is invalid")
            if workspace is None:
                # The slots the library's plan uses with room for all of them, within half of
                # the device memory that is free.
                order = (ctypes.c_int32 * G)()
                conc = ctypes.c_int32(0)
                st = lib.gptq_round_plan(self.arr, G, ctypes.c_size_t(self.slot_bytes * G),
                                         int(max_concurrency), order, ctypes.byref(conc))
                if st != GPTQ_OK:
                    raise GptqError(st, "gptq_round_plan")
                free = torch.cuda.mem_get_info(dev)[0]
                k = max(1, min(conc.value, free // 2 // self.slot_bytes))
                workspace = torch.empty(self.slot_bytes * k, dtype=torch.uint8, device=dev)
            else:
                _dev(workspace, torch.uint8, "workspace", align=256, device=dev)
        self.workspace = workspace
        self.max_concurrency = int(max_concurrency)

    def plan(self):
        """(order, concurrency) of the round as the library schedules it."""
        G = len(self.arr)
        order = (ctypes.c_int32 * G)()
        conc = ctypes.c_int32(0)
        st = load().gptq_round_plan(self.arr, G, self.workspace.numel(), self.max_concurrency,
                                    order, ctypes.byref(conc))
        if st != GPTQ_OK:
            raise GptqError(st, "gptq_round_plan")
        return list(order), conc.value

    def linear(self, X, group: int, member: int, bias=None, act="none", residual=None, out=None, workspace=None,
               stream=None, exact: bool = False):
        """:func:`gptq_linear` by a member's quantized weights, once the round has run: the layer's
        outputs, for the next layer's calibration inputs or a check."""
        codec = "q4tp" if self.arr[group].member[member].codec == CODEC["q4tp"] else "q2tp"
        _, _, codes, _, scale = self.results[group]["members"][member]
        return gptq_linear(X, codes, scale, codec, bias, act, residual, out, workspace, stream, exact)

    def gated(self, X, group: int, gate: int, up: int, act="silu", gate_bias=None, up_bias=None, out=None, workspace=None,
              stream=None, exact: bool = False):
        """:func:`gptq_gated` by two members' quantized weights (of one codec), once the round has run."""
        g, u = (self.arr[group].member[m].codec for m in (gate, up))
        if g != u:
            raise ValueError("the two members have different codecs")
        w = [(m[2], m[4]) for m in (self.results[group]["members"][k] for k in (gate, up))]
        return gptq_gated(X, *w, "q4tp" if g == CODEC["q4tp"] else "q2tp", act, gate_bias, up_bias, out, workspace, stream, exact)

    def run(self, stream=None) -> int:
        st = load().gptq_round(self.arr, len(self.arr), ctypes.c_void_p(self.workspace.data_ptr()),
                               self.workspace.numel(), self.max_concurrency, _stream(stream))
        for i, r in enumerate(self.results):
            r["status"] = int(self.arr[i].status)
            r["report"] = self.arr[i].report.as_dict()
        return int(st)


def gptq_round(groups, max_concurrency: int = 0, workspace=None, stream=None):
    """Run one batched round (see Round).  Returns (status, results)."""
    r = Round(groups, max_concurrency, workspace, stream)
    st = r.run(stream)
    return st, r.results


class check_mode:
    """Context manager: the library's calls run as dry runs of their schedule (no GPU; device
    pointers are never dereferenced) and return GPTQ_ECHECK when an access leaves its buffers
    or two launches on different streams race; see include/gptq_check.h."""

    def __enter__(self):
        load().gptq_check_mode(1)
        return self

    def __exit__(self, *exc):
        load().gptq_check_mode(0)
        return False


def check_message() -> str:
    return load().gptq_check_message().decode()


def check_selftest(which: int) -> int:
    return int(load().gptq_check_selftest(int(which)))


def check_tile_order(M: int, N: int, lower: bool) -> int:
    """Status of the host-side check of the tile GEMM's workgroup -> tile map for one shape."""
    return int(load().gptq_check_tile_order(int(M), int(N), 1 if lower else 0))


__all__ = ["check_mode", "check_message", "check_selftest", "check_tile_order", "gptq_gram_add", "gptq_debias",
           "gptq_act_order_perm", "gptq_permute_hessian", "gptq_sweep_act_order",
           "sweep_act_order_workspace_size", "gptq_ladder_q2", "gptq_sweep_q2",
           "gptq_sweep_act_order_q2", "gptq_debias_q2",
           "debias_workspace_size", "gptq_fold", "FOLD_PRECISION", "gptq_ladder", "gptq_sweep", "gptq_sweep_inplace", "fold_workspace_size",
           "sweep_workspace_size", "require_native", "load", "GptqError", "profile_enable",
           "profile_collect", "LIB_PATH", "gptq_round", "Round", "RoundGroup", "RoundMember", "CODEC",
           "gptq_linear", "linear_workspace_size", "gptq_cache_write", "gptq_cache_read", "gptq_cache_attention",
           "cache_alloc", "KVCache", "DTYPE", "ACT"]
