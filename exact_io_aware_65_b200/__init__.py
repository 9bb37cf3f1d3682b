"""Exact IO-aware attention (FlashAttention forward and backward) for B200.

A thin ctypes binding over ``libfa.so``: it only checks tensor properties and
marshals pointers, sizes and the CUDA stream into the C ABI declared in
``include/fa.h``.  Every step of the computation runs in the library's CUDA
kernels; there is no fallback path.  PyTorch supplies device memory and
streams.

    O, LSE = fa.fwd(Q, K, V, mask="causal", scale=d ** -0.5)
    dQ, dK, dV = fa.bwd(Q, K, V, O, dO, LSE, mask="causal", scale=d ** -0.5)

Tensors are bf16 [B, H, N, d] contiguous CUDA tensors, LSE is fp32 [B, H, N].
``block_mask`` (mask="block") is a uint8 [ceil(N/128), ceil(N/128)] CUDA
tensor shared by every batch and head.
"""
from __future__ import annotations

import ctypes
import os
import struct
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# FA_LIBRARY selects another build of the same library, e.g. the
# index-checking debug build libfa_debug.so.
LIB_PATH = os.environ.get("FA_LIBRARY") or os.path.join(_HERE, "libfa.so")

MASKS = {"none": 0, "causal": 1, "block": 2}
STATUS = {0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_CUDA",
          4: "FA_ERR_WORKSPACE", 5: "FA_ERR_TIMEOUT", 6: "FA_ERR_BOUNDS"}

# Every symbol include/fa.h declares, with its ctypes signature.
_vp, _i, _f, _sz, _u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_uint64
_i64 = ctypes.c_int64
SIGNATURES = {
    "fa_fwd": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _f, _vp, _vp, _vp]),
    "fa_bwd_workspace_size": (_sz, [_i, _i, _i, _i]),
    "fa_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _f, _vp, _vp, _vp, _vp, _sz, _vp]),
    "fa_bwd_stage": (_i, [_i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _f, _vp, _vp, _vp, _vp,
                          _sz, _vp]),
    "fa_fwd_qk": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _f, _vp, _vp, _vp]),
    "fa_bwd_workspace_size_qk": (_sz, [_i, _i, _i, _i, _i]),
    "fa_bwd_qk": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _f, _vp, _vp, _vp, _vp, _sz,
                       _vp]),
    "fa_bwd_qk_deterministic": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _f, _vp, _vp,
                                     _vp, _vp, _sz, _vp]),
    "fa_fwd_varlen": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _f, _vp, _vp, _vp, _vp, _vp]),
    "fa_bwd_varlen": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _f, _vp, _vp, _i, _vp, _vp,
                           _vp, _vp, _sz, _vp]),
    "fa_decode_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "fa_decode": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _sz, _vp]),
    "fa_fwd_packed_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "fa_fwd_packed": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _vp, _vp, _sz, _vp]),
    "fa_bwd_packed_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "fa_bwd_packed": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp, _vp,
                           _vp, _sz, _vp]),
    "fa_paged_append": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _vp]),
    "fa_paged_decode_workspace_size": (_sz, [_i, _i, _i, _i, _i64, _i]),
    "fa_paged_decode": (_i, [_vp, _vp, _i, _vp, _f, _vp, _i64, _i64, _i, _vp, _vp, _vp, _sz, _vp]),
    "fa_paged_evict": (_i, [_vp, _vp, _vp, _i64, _i, _vp, _i64, _i64, _i, _i, _vp, _i64, _i64, _i64, _vp, _vp, _vp]),
    "fa_standard_fwd_workspace_size": (_sz, [_i, _i, _i, _i]),
    "fa_standard_fwd": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _f, _vp, _vp, _vp, _sz, _vp]),
    "fa_bwd_static_workspace": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _f, _vp, _vp,
                                     _vp, _vp]),
    "fa_device_status": (_i, [_vp]),
    "fa_set_wait_timeout_ns": (None, [_u64]),
    "fa_status_string": (ctypes.c_char_p, [_i]),
    "fa_selftest_bounded_wait": (_i, [_u64, _vp]),
    "fa_selftest_mma_tile": (_i, [_vp, _vp, _vp, _i, _i, _i, _vp]),
}


# The structures of include/fa.h.  The calls below pass them as packed bytes (the
# same layout): filling a ctypes structure field by field takes longer than the
# smallest kernels.
_ROWS, _CACHE = struct.Struct("@Pqq"), struct.Struct("@PPiiiiiqqqPPPiiq")


class _Rows(ctypes.Structure):
    """fa_rows of include/fa.h."""
    _fields_ = [("data", _vp), ("row_stride", _i64), ("head_stride", _i64)]


class _PagedCache(ctypes.Structure):
    """fa_paged_cache of include/fa.h."""
    _fields_ = [("K", _vp), ("V", _vp), ("dtype", _i), ("num_pages", _i), ("page_size", _i), ("Hkv", _i), ("d", _i),
                ("page_stride", _i64), ("head_stride", _i64), ("row_stride", _i64), ("k_scale", _vp),
                ("v_scale", _vp), ("page_table", _vp), ("B", _i), ("max_pages", _i), ("table_stride", _i64)]


class _Cache:
    """A checked cache: its packed fa_paged_cache, and the sizes that the calls go by."""
    __slots__ = ("c", "B", "Hkv", "d", "max_pages", "page_size")

    def __init__(self, c, B, Hkv, d, max_pages, page_size):
        self.c, self.B, self.Hkv, self.d, self.max_pages, self.page_size = c, B, Hkv, d, max_pages, page_size


class FAError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {STATUS.get(code, code)}")
        self.code = code


_lib = None
# The packed and paged calls of _binding.so (csrc/binding.cpp): the same checks
# and the same library, without ctypes.  What it does not take (it answers None)
# goes through the Python code of the call.
_fast = None


def lib() -> ctypes.CDLL:
    """Load libfa.so (build it first with ``python -m exact_io_aware_65_b200.build``)."""
    global _lib, _fast
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise FAError(3, f"CUDA library missing at {LIB_PATH}; build it with "
                             "`python -m exact_io_aware_65_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
        if os.path.exists(os.path.join(_HERE, "_binding.so")):
            try:
                from . import _binding

                _binding.use(L._handle)
                _fast = _binding
            except ImportError as e:  # built against another torch
                warnings.warn(f"_binding.so does not load ({e}); calls go through ctypes. Rebuild it with "
                              "`python -m exact_io_aware_65_b200.build`")
    return _lib


def _check(code: int, what: str):
    if code != 0:
        raise FAError(code, what)


def _taken(answer, what: str) -> bool:
    """Whether ``_fast`` made the call; its status, if the library refused."""
    if answer.__class__ is int:
        raise FAError(answer, what)
    return answer is not None


def _stream(stream) -> int:
    if stream is None:  # the current device's current stream, without building a Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _mask(mask, block_mask, nbq=None, nbk=None, device=None):
    """Mask kind and block-mask pointer.  The kernels read a row-major
    [nbq, nbk] uint8 grid, so a block mask must hold exactly that many
    entries, contiguous, on the inputs' device."""
    kind = MASKS[mask] if isinstance(mask, str) else int(mask)
    ptr = None
    if kind == MASKS["block"]:
        if block_mask is None or not block_mask.is_cuda or block_mask.dtype != torch.uint8:
            raise FAError(1, "block mask must be a uint8 CUDA tensor")
        if not block_mask.is_contiguous():
            raise FAError(1, "block mask must be contiguous")
        if nbq is not None and block_mask.numel() != nbq * nbk:
            raise FAError(1, f"block mask must hold {nbq} x {nbk} entries (128-row query tiles by "
                             f"128-key tiles), got {tuple(block_mask.shape)}")
        if device is not None and block_mask.device != device:
            raise FAError(1, f"block mask must be on {device}")
        ptr = block_mask.data_ptr()
    return kind, ptr


def _tiles(n):
    return (n + 127) // 128


def _check_buf(t, name, shape, dtype, device):
    """A caller-supplied tensor the kernels read or write through a raw
    pointer: it must have exactly the size the call implies, be contiguous
    and sit on the inputs' device."""
    if not isinstance(t, torch.Tensor):
        raise FAError(1, f"{name} must be a tensor")
    if t.device != device or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise FAError(1, f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}" + ("" if t.is_contiguous() else
                                                                       " (not contiguous)"))
    return t


def _workspace(ws, need, device):
    """Device pointer and size in bytes of a caller-supplied workspace."""
    if not isinstance(ws, torch.Tensor) or ws.device != device or not ws.is_contiguous():
        raise FAError(4, f"workspace must be a contiguous tensor on {device}")
    nbytes = ws.numel() * ws.element_size()
    if nbytes < need:
        raise FAError(4, f"workspace holds {nbytes} bytes, the call needs {need}")
    return ws.data_ptr(), nbytes


def _check_qkv(*ts):
    for t in ts:
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()
                and t.dim() == 4):
            raise FAError(1, "tensors must be contiguous bf16 CUDA tensors [B, H, N, d]")
    if any(t.device != ts[0].device for t in ts):
        raise FAError(1, "all tensors must be on one device")


def _nk(Q, K, V):
    """Key count of K, V [B,H,Nk,d] (heads and head dimension as Q's)."""
    if K.shape != V.shape or K.shape[:2] != Q.shape[:2] or K.shape[3] != Q.shape[3]:
        raise FAError(1, "K and V must be [B, H, Nk, d] with Q's B, H and d")
    return K.shape[2]


def _lens(t, B, device):
    """Device pointer of an optional per-batch-element length vector."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.device == device and t.dtype == torch.int32 and t.is_contiguous()
            and t.numel() == B):
        raise FAError(1, f"sequence lengths must be a contiguous int32 tensor [B] on {device}")
    return t.data_ptr()


def _outputs(Q, N, O, LSE):
    """O [B,H,N,d] bf16 and LSE [B,H,N] fp32: the caller's, checked, or new."""
    B, H, _, d = Q.shape
    O = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=Q.device) if O is None else \
        _check_buf(O, "O", (B, H, N, d), torch.bfloat16, Q.device)
    LSE = torch.empty((B, H, N), dtype=torch.float32, device=Q.device) if LSE is None else \
        _check_buf(LSE, "LSE", (B, H, N), torch.float32, Q.device)
    return O, LSE


def fwd(Q, K, V, mask="none", block_mask=None, scale=None, O=None, LSE=None, stream=None, seqlens_q=None,
        seqlens_k=None):
    """O [B,H,Nq,d] bf16 and LSE [B,H,Nq] fp32 (natural log); K, V are
    [B,H,Nk,d] (Nk may differ from Nq: fa_fwd_qk)."""
    _check_qkv(Q, K, V)
    B, H, N, d = Q.shape
    Nk = _nk(Q, K, V)
    scale = d ** -0.5 if scale is None else float(scale)
    kind, mptr = _mask(mask, block_mask, _tiles(N), _tiles(Nk), Q.device)
    O, LSE = _outputs(Q, N, O, LSE)
    if seqlens_q is not None or seqlens_k is not None:
        _check(lib().fa_fwd_varlen(Q.data_ptr(), K.data_ptr(), V.data_ptr(), B, H, N, Nk, d, kind, mptr, scale,
                                   _lens(seqlens_q, B, Q.device), _lens(seqlens_k, B, Q.device), O.data_ptr(),
                                   LSE.data_ptr(), _stream(stream)), "fa_fwd_varlen")
    elif Nk == N:
        _check(lib().fa_fwd(Q.data_ptr(), K.data_ptr(), V.data_ptr(), B, H, N, d, kind, mptr, scale,
                            O.data_ptr(), LSE.data_ptr(), _stream(stream)), "fa_fwd")
    else:
        _check(lib().fa_fwd_qk(Q.data_ptr(), K.data_ptr(), V.data_ptr(), B, H, N, Nk, d, kind, mptr, scale,
                               O.data_ptr(), LSE.data_ptr(), _stream(stream)), "fa_fwd_qk")
    return O, LSE


def bwd_workspace_size(B, H, N, d, Nk=None) -> int:
    if Nk is None:
        return int(lib().fa_bwd_workspace_size(B, H, N, d))
    return int(lib().fa_bwd_workspace_size_qk(B, H, N, Nk, d))


def _bwd_buffers(Q, K, V, O, dO, LSE, dQ, dK, dV):
    """Checks the backward's inputs beyond Q, K, V and returns its outputs."""
    _check_qkv(Q, K, V, O, dO)
    B, H, N, d = Q.shape
    Nk = _nk(Q, K, V)
    _check_buf(O, "O", Q.shape, torch.bfloat16, Q.device)
    _check_buf(dO, "dO", Q.shape, torch.bfloat16, Q.device)
    _check_buf(LSE, "LSE", (B, H, N), torch.float32, Q.device)
    dQ = torch.empty_like(Q) if dQ is None else _check_buf(dQ, "dQ", Q.shape, torch.bfloat16, Q.device)
    dK = torch.empty_like(K) if dK is None else _check_buf(dK, "dK", K.shape, torch.bfloat16, Q.device)
    dV = torch.empty_like(V) if dV is None else _check_buf(dV, "dV", V.shape, torch.bfloat16, Q.device)
    return Nk, dQ, dK, dV


def bwd(Q, K, V, O, dO, LSE, mask="none", block_mask=None, scale=None, dQ=None, dK=None, dV=None,
        workspace=None, stream=None, deterministic=False, seqlens_q=None, seqlens_k=None):
    """dQ [B,H,Nq,d], dK, dV [B,H,Nk,d] bf16 (Nk may differ from Nq: fa_bwd_qk)."""
    Nk, dQ, dK, dV = _bwd_buffers(Q, K, V, O, dO, LSE, dQ, dK, dV)
    B, H, N, d = Q.shape
    scale = d ** -0.5 if scale is None else float(scale)
    kind, mptr = _mask(mask, block_mask, _tiles(N), _tiles(Nk), Q.device)
    need = bwd_workspace_size(B, H, N, d, Nk)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
    wptr, wbytes = _workspace(workspace, need, Q.device)
    if seqlens_q is not None or seqlens_k is not None:
        _check(lib().fa_bwd_varlen(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), dO.data_ptr(),
                                   LSE.data_ptr(), B, H, N, Nk, d, kind, mptr, scale,
                                   _lens(seqlens_q, B, Q.device), _lens(seqlens_k, B, Q.device),
                                   1 if deterministic else 0, dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), wptr,
                                   wbytes, _stream(stream)), "fa_bwd_varlen")
    elif deterministic:
        _check(lib().fa_bwd_qk_deterministic(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), dO.data_ptr(),
                                             LSE.data_ptr(), B, H, N, Nk, d, kind, mptr, scale, dQ.data_ptr(),
                                             dK.data_ptr(), dV.data_ptr(), wptr, wbytes, _stream(stream)),
               "fa_bwd_qk_deterministic")
    elif Nk == N:
        _check(lib().fa_bwd(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), dO.data_ptr(),
                            LSE.data_ptr(), B, H, N, d, kind, mptr, scale, dQ.data_ptr(), dK.data_ptr(),
                            dV.data_ptr(), wptr, wbytes, _stream(stream)), "fa_bwd")
    else:
        _check(lib().fa_bwd_qk(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), dO.data_ptr(),
                               LSE.data_ptr(), B, H, N, Nk, d, kind, mptr, scale, dQ.data_ptr(), dK.data_ptr(),
                               dV.data_ptr(), wptr, wbytes, _stream(stream)), "fa_bwd_qk")
    return dQ, dK, dV


def bwd_stage(stage, Q, K, V, O, dO, LSE, dQ, dK, dV, workspace, mask="none", block_mask=None,
              scale=None, stream=None):
    """One of the three launches of ``bwd`` (0: prep, 1: main, 2: dQ
    convert); running 0, 1, 2 in order on one workspace equals ``bwd``.
    Self-attention only (K, V with Q's sequence length)."""
    Nk, dQ, dK, dV = _bwd_buffers(Q, K, V, O, dO, LSE, dQ, dK, dV)
    B, H, N, d = Q.shape
    if Nk != N:
        raise FAError(1, "bwd_stage takes K and V with Q's sequence length")
    scale = d ** -0.5 if scale is None else float(scale)
    kind, mptr = _mask(mask, block_mask, _tiles(N), _tiles(N), Q.device)
    wptr, wbytes = _workspace(workspace, bwd_workspace_size(B, H, N, d), Q.device)
    _check(lib().fa_bwd_stage(int(stage), Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
                              dO.data_ptr(), LSE.data_ptr(), B, H, N, d, kind, mptr, scale, dQ.data_ptr(),
                              dK.data_ptr(), dV.data_ptr(), wptr, wbytes, _stream(stream)), f"fa_bwd_stage({stage})")


def bwd_static_workspace(Q, K, V, O, dO, LSE, mask="none", block_mask=None, scale=None, dQ=None, dK=None,
                         dV=None, stream=None):
    """``bwd`` with the library's own fixed device scratch instead of a
    workspace (fa_bwd_static_workspace): allocates no workspace; calls whose
    kernels overlap on one device must not use it concurrently."""
    Nk, dQ, dK, dV = _bwd_buffers(Q, K, V, O, dO, LSE, dQ, dK, dV)
    B, H, N, d = Q.shape
    if Nk != N:
        raise FAError(1, "bwd_static_workspace takes K and V with Q's sequence length")
    scale = d ** -0.5 if scale is None else float(scale)
    kind, mptr = _mask(mask, block_mask, _tiles(N), _tiles(N), Q.device)
    _check(lib().fa_bwd_static_workspace(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), dO.data_ptr(),
                                         LSE.data_ptr(), B, H, N, d, kind, mptr, scale, dQ.data_ptr(),
                                         dK.data_ptr(), dV.data_ptr(), _stream(stream)), "fa_bwd_static_workspace")
    return dQ, dK, dV


def decode(Q, K, V, mask="none", scale=None, O=None, LSE=None, workspace=None, stream=None):
    """Decode against a KV cache: Q [B,H,Nq,d] (Nq <= 16) against K, V
    [B,H,Nk,d]; returns O [B,H,Nq,d] bf16 and LSE [B,H,Nq] fp32."""
    _check_qkv(Q, K, V)
    B, H, N, d = Q.shape
    Nk = _nk(Q, K, V)
    scale = d ** -0.5 if scale is None else float(scale)
    kind = MASKS[mask] if isinstance(mask, str) else int(mask)
    if kind == MASKS["block"]:
        raise FAError(2, "decode takes no block mask")
    O, LSE = _outputs(Q, N, O, LSE)
    need = decode_workspace_size(B, H, N, Nk, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
    wptr, wbytes = _workspace(workspace, need, Q.device)
    _check(lib().fa_decode(Q.data_ptr(), K.data_ptr(), V.data_ptr(), B, H, N, Nk, d, kind, scale, O.data_ptr(),
                           LSE.data_ptr(), wptr, wbytes, _stream(stream)), "fa_decode")
    return O, LSE


# ---- packed rows and the paged cache -----------------------------------------
def _run(name, device, stream, *args):
    """Call ``name`` with ``device`` current (its kernels launch there) on
    ``stream``, by default that device's current stream."""
    if device.index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            code = getattr(lib(), name)(*args, _stream(stream))
    else:
        code = getattr(_lib or lib(), name)(*args, _stream(stream))
    if code:
        raise FAError(code, name)


def _empty(shape, dtype, device, stream, like=None):
    """A new buffer for a call on ``stream``: the allocator hands memory out in
    the order of the stream it is asked on, so that must be the call's.
    ``like``: a tensor that has the shape and type, if it happens to be
    contiguous (a cheaper call)."""
    if stream is None:
        if like is not None and like.is_contiguous():
            return torch.empty_like(like)
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


_BF16, _E4M3 = torch.bfloat16, torch.float8_e4m3fn


def _rows(t, name, heads=None, d=None, rows=None, device=None):
    """fa_rows of a bf16 CUDA tensor [rows, heads, d] whose last dimension is
    contiguous; the rows and heads may be strided."""
    try:
        n, h, w = t.shape
        rs, hs, ds = t.stride()
        ptr = t.data_ptr()
        good = t.dtype is _BF16 and t.is_cuda
    except (AttributeError, ValueError, TypeError, RuntimeError):
        good = False
    if not good:
        raise FAError(1, f"{name} must be a bf16 CUDA tensor [rows, heads, d]")
    if (heads is not None and h != heads) or (d is not None and w != d) or (rows is not None and n != rows):
        raise FAError(1, f"{name} must be [{'rows' if rows is None else rows}, {'heads' if heads is None else heads}, "
                         f"{'d' if d is None else d}], got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise FAError(1, f"{name} must be on {device}, got {t.device}")
    if n <= 1:  # the stride of a single row or head is never used
        rs = h * w
    if h <= 1:
        hs = w
    if (ds != 1 and w > 1) or (rs | hs) & 7 or ptr & 15:
        raise FAError(1, f"{name}: d must be contiguous, and rows and heads start on 16-byte boundaries (strides "
                         f"{t.stride()})")
    return _ROWS.pack(ptr, rs, hs)


def _int32(t, name, n, device):
    """Device pointer of a contiguous int32 vector [n]."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.shape == (n,) and t.device == device
            and t.is_contiguous()):
        raise FAError(1, f"{name} must be a contiguous int32 tensor [{n}] on {device}")
    return t.data_ptr()


def _sequences(cu):
    """Number of sequences that an int32 vector of first rows [B + 1] describes."""
    if not (isinstance(cu, torch.Tensor) and cu.dim() == 1 and cu.shape[0] >= 2):
        raise FAError(1, "cu_q must be an int32 tensor [B + 1] with B >= 1")
    return cu.shape[0] - 1


def _table(t, name, device):
    """Pointer, width and row stride of a page table [B, pages] (int32)."""
    if not (isinstance(t, torch.Tensor) and t.device == device and t.dtype == torch.int32 and t.dim() == 2
            and t.shape[0] > 0 and t.shape[1] > 0 and (t.stride(1) == 1 or t.shape[1] == 1)):
        raise FAError(1, f"{name} must be an int32 tensor [B, pages] on {device} with contiguous rows")
    return t.data_ptr(), t.shape[1], t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _packed_mask(mask):
    kind = MASKS[mask] if isinstance(mask, str) else int(mask)
    if kind == MASKS["block"]:
        raise FAError(2, "packed attention takes no block mask")
    return kind


def fwd_packed_workspace_size(B, Tq, Hq, Hkv, d) -> int:
    return int(lib().fa_fwd_packed_workspace_size(B, Tq, Hq, Hkv, d))


def fwd_packed(Q, K, V, cu_q, cu_k, mask="none", scale=None, O=None, LSE=None, workspace=None, stream=None):
    """Attention over packed sequences with grouped heads: Q [Tq, Hq, d], K, V
    [Tk, Hkv, d] bf16 (rows and heads may be strided), sequence b in rows
    cu_q[b] .. cu_q[b + 1] of Q and cu_k[b] .. cu_k[b + 1] of K and V (int32
    [B + 1]); mask "none" or "causal" (aligned at each sequence's last query and
    key).  Returns O [Tq, Hq, d] bf16 and LSE [Hq, Tq] fp32; rows that belong to
    no sequence are not written."""
    kind = _packed_mask(mask)
    if _fast is not None and stream is None:
        made = _fast.fwd_packed(Q, K, V, cu_q, cu_k, O, LSE, workspace, kind, scale)
        if _taken(made, "fa_fwd_packed"):
            return made
    q = _rows(Q, "Q")
    dev = Q.device
    Tq, Hq, d = Q.shape
    k = _rows(K, "K", None, d, None, dev)
    Tk, Hkv, _ = K.shape
    v = _rows(V, "V", Hkv, d, Tk, dev)
    B = _sequences(cu_q)
    scale = d ** -0.5 if scale is None else float(scale)
    if O is None:
        O = _empty((Tq, Hq, d), _BF16, dev, stream, Q)
    o = _rows(O, "O", Hq, d, Tq, dev)
    LSE = _empty((Hq, Tq), torch.float32, dev, stream) if LSE is None else \
        _check_buf(LSE, "LSE", (Hq, Tq), torch.float32, dev)
    need = fwd_packed_workspace_size(B, Tq, Hq, Hkv, d)
    if workspace is None and need:
        workspace = _empty(need, torch.uint8, dev, stream)
    wp, wn = (None, 0) if workspace is None else _workspace(workspace, need, dev)
    _run("fa_fwd_packed", dev, stream, q, k, v,
         _int32(cu_q, "cu_q", B + 1, dev), _int32(cu_k, "cu_k", B + 1, dev), B, Tq, Tk, Hq, Hkv, d, kind,
         scale, o, LSE.data_ptr(), wp, wn)
    return O, LSE


def bwd_packed_workspace_size(B, Tq, Tk, Hq, Hkv, d) -> int:
    return int(lib().fa_bwd_packed_workspace_size(B, Tq, Tk, Hq, Hkv, d))


def bwd_packed(Q, K, V, O, dO, LSE, cu_q, cu_k, mask="none", scale=None, dQ=None, dK=None, dV=None, workspace=None,
               stream=None, deterministic=False):
    """The gradients of ``fwd_packed``: dQ [Tq, Hq, d], dK, dV [Tk, Hkv, d]
    (summed over each key head's query heads) from O and LSE of the forward
    with the same mask and scale."""
    kind = _packed_mask(mask)
    if _fast is not None and stream is None:
        made = _fast.bwd_packed(Q, K, V, cu_q, cu_k, O, dO, LSE, dQ, dK, dV, workspace, kind, scale, 1 if deterministic else 0)
        if _taken(made, "fa_bwd_packed"):
            return made
    q = _rows(Q, "Q")
    dev = Q.device
    Tq, Hq, d = Q.shape
    k = _rows(K, "K", None, d, None, dev)
    Tk, Hkv, _ = K.shape
    v = _rows(V, "V", Hkv, d, Tk, dev)
    o, g = _rows(O, "O", Hq, d, Tq, dev), _rows(dO, "dO", Hq, d, Tq, dev)
    _check_buf(LSE, "LSE", (Hq, Tq), torch.float32, dev)
    B = _sequences(cu_q)
    scale = d ** -0.5 if scale is None else float(scale)
    if dQ is None:
        dQ = _empty((Tq, Hq, d), _BF16, dev, stream, Q)
    if dK is None:
        dK = _empty((Tk, Hkv, d), _BF16, dev, stream, K)
    if dV is None:
        dV = _empty((Tk, Hkv, d), _BF16, dev, stream, V)
    dq, dk, dv = _rows(dQ, "dQ", Hq, d, Tq, dev), _rows(dK, "dK", Hkv, d, Tk, dev), _rows(dV, "dV", Hkv, d, Tk, dev)
    need = bwd_packed_workspace_size(B, Tq, Tk, Hq, Hkv, d)
    if workspace is None:
        workspace = _empty(need, torch.uint8, dev, stream)
    wp, wn = _workspace(workspace, need, dev)
    _run("fa_bwd_packed", dev, stream, q, k, v, o, g,
         LSE.data_ptr(), _int32(cu_q, "cu_q", B + 1, dev), _int32(cu_k, "cu_k", B + 1, dev), B, Tq, Tk, Hq, Hkv, d,
         kind, scale, 1 if deterministic else 0, dq, dk, dv, wp, wn)
    return dQ, dK, dV


def _paged_cache(k_cache, v_cache, page_table, k_scale=None, v_scale=None, scales=True):
    """fa_paged_cache of two pools [pages, Hkv, page_size, d]."""
    for t in (k_cache, v_cache):
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dim() == 4 and (t.dtype is _BF16 or t.dtype is _E4M3)):
            raise FAError(1, "cache pools must be bf16 or float8_e4m3fn CUDA tensors [pages, Hkv, page_size, d]")
    dev = k_cache.device
    pages, Hkv, page, d = k_cache.shape
    sp, sh, sr, sd = strides = k_cache.stride()
    if (v_cache.shape != k_cache.shape or v_cache.dtype is not k_cache.dtype or v_cache.device != dev
            or v_cache.stride() != strides):
        raise FAError(1, "the K and V pools must have one shape, type, device and layout")
    eight = k_cache.dtype is _E4M3
    # (the stride of a dimension of one entry is never used)
    sp, sh, sr = sp if pages > 1 else 0, sh if Hkv > 1 else 0, sr if page > 1 else 0
    kp, vp = k_cache.data_ptr(), v_cache.data_ptr()
    if (sd != 1 and d > 1) or (sp | sh | sr) & (15 if eight else 7) or (kp | vp) & 15:
        raise FAError(1, "cache rows must be contiguous and start on 16-byte boundaries")
    ks = vs = 0
    if eight and scales:
        ks = _check_buf(k_scale, "k_scale", (Hkv,), torch.float32, dev).data_ptr()
        vs = _check_buf(v_scale, "v_scale", (Hkv,), torch.float32, dev).data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise FAError(1, "k_scale and v_scale belong to float8_e4m3fn pools")
    tp, width, ts = _table(page_table, "page_table", dev)
    B = page_table.shape[0]
    return _Cache(_CACHE.pack(kp, vp, 1 if eight else 0, pages, page, Hkv, d, sp, sh, sr, ks, vs, tp, B, width, ts), B,
                  Hkv, d, width, page)


def _weights(t, name, B, Hkv, least, device):
    """Pointer and strides of fp32 weights [B, Hkv, >= least]."""
    if not (isinstance(t, torch.Tensor) and t.device == device and t.dtype == torch.float32 and t.dim() == 3
            and tuple(t.shape[:2]) == (B, Hkv) and t.shape[2] >= least and (t.stride(2) == 1 or t.shape[2] == 1)):
        raise FAError(1, f"{name} must be an fp32 tensor [{B}, {Hkv}, at least {least}] on {device} with contiguous rows")
    return t.data_ptr(), t.stride(0) if B > 1 else 0, t.stride(1) if Hkv > 1 else 0


def paged_append(K, V, cu_seqlens, lens, k_cache, v_cache, page_table, k_scale=None, v_scale=None, stream=None):
    """Write the packed rows K, V [T, Hkv, d] (bf16) into the paged cache: row
    t of sequence b (cu_seqlens[b] <= t < cu_seqlens[b + 1], int32 [B + 1])
    goes to position lens[b] + t - cu_seqlens[b]; ``lens`` (int32 [B]) counts
    the positions already held and is not changed.  Pools are
    [pages, Hkv, page_size, d], bf16 or float8_e4m3fn (then with fp32 scales
    [Hkv]); page_table is int32 [B, pages]."""
    if _fast is not None and stream is None:
        if _taken(_fast.paged_append(K, V, cu_seqlens, lens, k_cache, v_cache, page_table, k_scale, v_scale), "fa_paged_append"):
            return
    c = _paged_cache(k_cache, v_cache, page_table, k_scale, v_scale)
    dev = k_cache.device
    k = _rows(K, "K", c.Hkv, c.d, device=dev)
    v = _rows(V, "V", c.Hkv, c.d, K.shape[0], dev)
    _run("fa_paged_append", dev, stream, c.c, k, v,
         _int32(cu_seqlens, "cu_seqlens", c.B + 1, dev), _int32(lens, "lens", c.B, dev), K.shape[0])


def paged_decode_workspace_size(B, Hq, Hkv, d, max_len, weights=False) -> int:
    """Bytes for ``paged_decode``; max_len is the page table's width times the
    page size."""
    return int(lib().fa_paged_decode_workspace_size(B, Hq, Hkv, d, max_len, 1 if weights else 0))


def paged_decode(Q, k_cache, v_cache, page_table, lens, scale=None, k_scale=None, v_scale=None, weights=None,
                 accumulate=False, O=None, LSE=None, workspace=None, stream=None):
    """One new token per sequence over its cached keys, grouped heads: Q
    [B, Hq, d] bf16 against the first lens[b] positions of the paged cache;
    returns O [B, Hq, d] bf16 and LSE [B, Hq] fp32.  ``weights`` (fp32
    [B, Hkv, at least pages * page_size]) receives the attention that each key
    drew, summed over its group of query heads, or is raised by it with
    ``accumulate``."""
    if _fast is not None and stream is None:
        made = _fast.paged_decode(Q, k_cache, v_cache, page_table, lens, k_scale, v_scale, weights, O, LSE, workspace, scale,
                                  1 if accumulate else 0)
        if _taken(made, "fa_paged_decode"):
            return made
    c = _paged_cache(k_cache, v_cache, page_table, k_scale, v_scale)
    dev, B, d = k_cache.device, c.B, c.d
    q = _rows(Q, "Q", None, d, B, dev)
    Hq = Q.shape[1]
    cap = c.max_pages * c.page_size
    scale = d ** -0.5 if scale is None else float(scale)
    lp = _int32(lens, "lens", B, dev)
    wp = wb = wh = 0
    if weights is not None:
        wp, wb, wh = _weights(weights, "weights", B, c.Hkv, cap, dev)
    O = _empty((B, Hq, d), _BF16, dev, stream, Q) if O is None else _check_buf(O, "O", (B, Hq, d), _BF16, dev)
    LSE = _empty((B, Hq), torch.float32, dev, stream) if LSE is None else \
        _check_buf(LSE, "LSE", (B, Hq), torch.float32, dev)
    need = paged_decode_workspace_size(B, Hq, c.Hkv, d, cap, weights is not None)
    if workspace is None:
        workspace = _empty(need, torch.uint8, dev, stream)
    sp, sn = _workspace(workspace, need, dev)
    _run("fa_paged_decode", dev, stream, c.c, q, Hq, lp, scale, wp or None, wb, wh,
         1 if accumulate else 0, O.data_ptr(), LSE.data_ptr(), sp, sn)
    return O, LSE


def paged_evict(weights, k_cache, v_cache, page_table, lens, table_out, budget, recent, weights_out, kept=None,
                lens_out=None, stream=None):
    """Cut each sequence's cache to ``budget`` rows a head: the last ``recent``
    and the others of largest weight, copied in order to the pages of
    ``table_out`` (int32 [B, pages], pages of the same pools that no sequence
    of the call reads).  Returns kept [B, Hkv, budget] int32 (the positions
    kept, then -1) and lens_out [B] int32; ``weights_out`` (fp32
    [B, Hkv, width]) gets the kept rows' weights, then zeros.  Nothing is
    written in place: ``weights_out`` is not ``weights``, ``lens_out`` not
    ``lens``, and ``table_out`` not ``page_table``."""
    if _fast is not None and stream is None:
        made = _fast.paged_evict(weights, k_cache, v_cache, page_table, lens, table_out, weights_out, kept, lens_out, budget, recent)
        if _taken(made, "fa_paged_evict"):
            return made
    c = _paged_cache(k_cache, v_cache, page_table, scales=False)  # 8-bit rows move as they are
    dev, B, Hkv = k_cache.device, c.B, c.Hkv
    cap = c.max_pages * c.page_size
    wp, wb, wh = _weights(weights, "weights", B, Hkv, cap, dev)
    op, ob, oh = _weights(weights_out, "weights_out", B, Hkv, min(int(budget), cap), dev)
    tp, width, ts = _table(table_out, "table_out", dev)
    if table_out.shape[0] != B:
        raise FAError(1, f"table_out must have {B} rows")
    lp = _int32(lens, "lens", B, dev)
    budget, recent = int(budget), int(recent)
    if budget <= 0 or not 0 <= recent <= budget:
        raise FAError(1, "paged_evict takes budget > 0 and 0 <= recent <= budget")
    kept = _empty((B, Hkv, budget), torch.int32, dev, stream) if kept is None else \
        _check_buf(kept, "kept", (B, Hkv, budget), torch.int32, dev)
    lens_out = _empty((B,), torch.int32, dev, stream) if lens_out is None else \
        _check_buf(lens_out, "lens_out", (B,), torch.int32, dev)
    _run("fa_paged_evict", dev, stream, c.c, lp, tp, ts, width, wp, wb, wh, budget, recent, op, ob, oh,
         weights_out.shape[2], kept.data_ptr(), lens_out.data_ptr())
    return kept, lens_out


def standard_fwd(Q, K, V, mask="none", block_mask=None, scale=None, O=None, LSE=None, workspace=None,
                 stream=None):
    """Standard (materialising) attention, the baseline: O [B,H,N,d] bf16 and
    LSE [B,H,N] fp32, through an N x N score grid in HBM."""
    _check_qkv(Q, K, V)
    B, H, N, d = Q.shape
    if _nk(Q, K, V) != N:
        raise FAError(1, "standard_fwd takes K and V with Q's sequence length")
    scale = d ** -0.5 if scale is None else float(scale)
    kind, mptr = _mask(mask, block_mask, _tiles(N), _tiles(N), Q.device)
    O, LSE = _outputs(Q, N, O, LSE)
    need = standard_fwd_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
    wptr, wbytes = _workspace(workspace, need, Q.device)
    _check(lib().fa_standard_fwd(Q.data_ptr(), K.data_ptr(), V.data_ptr(), B, H, N, d, kind, mptr, scale,
                                 O.data_ptr(), LSE.data_ptr(), wptr, wbytes, _stream(stream)), "fa_standard_fwd")
    return O, LSE


def standard_fwd_workspace_size(B, H, N, d) -> int:
    return int(lib().fa_standard_fwd_workspace_size(B, H, N, d))


def decode_workspace_size(B, H, Nq, Nk, d) -> int:
    return int(lib().fa_decode_workspace_size(B, H, Nq, Nk, d))


def device_status(stream=None) -> int:
    """Synchronise and read/clear the device status word (0 = ok, 5 = timeout)."""
    return int(lib().fa_device_status(_stream(stream)))


def set_wait_timeout_ns(ns: int):
    lib().fa_set_wait_timeout_ns(int(ns))


def selftest_bounded_wait(timeout_ns: int, stream=None):
    _check(lib().fa_selftest_bounded_wait(int(timeout_ns), _stream(stream)), "fa_selftest_bounded_wait")


def selftest_mma_tile(A, B, n, k, mode, stream=None):
    """C [128, n] fp32 = A [128, k] times Bt^T with Bt [n, k] (mode 0), or
    times B [k, n] (mode 1), on one tensor-core tile."""
    if not (isinstance(A, torch.Tensor) and A.is_cuda):
        raise FAError(1, "A must be a CUDA tensor")
    _check_buf(A, "A", (128, k), torch.bfloat16, A.device)
    _check_buf(B, "B", (n, k) if mode == 0 else (k, n), torch.bfloat16, A.device)
    C = torch.empty((128, n), dtype=torch.float32, device=A.device)
    _check(lib().fa_selftest_mma_tile(A.data_ptr(), B.data_ptr(), C.data_ptr(), n, k, mode, _stream(stream)),
           "fa_selftest_mma_tile")
    return C
