"""GB300-native (sm_103a) MLA paged decode: a thin Python binding over the
C ABI in ``include/mla_decode.h``.

The three calls of one decode step of a Multi-head Latent Attention layer:

    o, lse = attend(q, kv, pages, indptr, scale, kv_scale, num_splits, split_tokens)
    latent, lse_merged = merge(o, lse)
    out = value_gate(latent, w_uv, gate, lengths, qlen)

and the operators around them: ``kv_append``, ``add_rms_norm``, ``norm_rope``
and ``query_absorb`` in front of attend, ``index_scores`` / ``index_select``
for attention to chosen tokens only, ``token_weights`` / ``kv_evict`` and
``value_gate_lora``.

This module only marshals arguments (for the operators but ``kv_append``
through a compiled module, ``csrc/binding.cpp``): it checks dtypes / shapes, allocates
outputs with torch (device memory), passes raw pointers and the current CUDA
stream to the native library, and turns error codes into exceptions.  Every
step of the computation runs in the library's CUDA kernels; there is no
fallback.  If the library has not been built (``build()``), every call
raises.
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import build as _build

D_QK, D_LATENT, D_V = 576, 512, 128
MLA_OK, MLA_ERR_INVALID, MLA_ERR_UNSUPPORTED, MLA_ERR_CUDA = 0, -1, -2, -3
ATTEND_CAUSAL, ATTEND_Q_FP8 = 1, 2
DEV_BAD_PAGE, DEV_BAD_INDPTR, DEV_TIMEOUT, DEV_BAD_PLAN, DEV_BAD_ADAPTER, DEV_BAD_POSITION = 1, 2, 4, 8, 16, 32
STATIC_SCRATCH_BYTES = 32 << 20   # MLA_STATIC_SCRATCH_BYTES: the partials buffer of decode_step_static

__all__ = ["Prepared", "attend", "merge", "value_gate", "merge_value_gate", "decode_step", "decode_step_static",
           "STATIC_SCRATCH_BYTES", "choose_splits", "plan_units", "debug_gather",
           "debug_wait_timeout", "debug_attend_mma",
           "kv_append", "norm_rope", "query_absorb", "index_scores", "index_select", "index_select_capacity",
           "add_rms_norm", "token_weights", "kv_evict", "value_gate_lora", "value_gate_lora_workspace",
           "token_weights_workspace", "device_status", "build", "library", "MlaError"]


class MlaError(RuntimeError):
    """A non-zero status from the native library."""

    def __init__(self, status: int, where: str, detail: str):
        super().__init__("%s failed: %s (%d)%s" % (where, _status_name(status), status,
                                                  ": " + detail if detail else ""))
        self.status = status


_lib = None


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the CUDA library in-tree (sm_103a) and return its path."""
    return _build.build(force=force, verbose=verbose)


def library() -> ctypes.CDLL:
    """The loaded native library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if not os.path.exists(path):
        raise RuntimeError("mla_decode_paged_gb300: native library %s is missing; run "
                           "mla_decode_paged_gb300.build() first (no CPU fallback exists)" % path)
    lib = ctypes.CDLL(path)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    lib.mla_decode_attend.argtypes = [vp, i64, vp, i64, vp, i64, vp, i32, i32, i32, f32, f32, i32, i32,
                                      vp, vp, vp]
    lib.mla_decode_attend_ex.argtypes = [vp, i64, vp, i64, vp, i64, vp, i32, i32, i32, f32, f32, i32, i32,
                                         vp, vp, ctypes.c_uint, vp]
    lib.mla_decode_attend_paged.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, i32, i32, i32, i32, f32, f32,
                                            i32, i32, vp, vp, ctypes.c_uint, vp]
    lib.mla_decode_attend_planned.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, i32, i32, i32, i32, f32, f32,
                                              f32, i32, i32, vp, vp, ctypes.c_uint, vp, i64, vp]
    lib.mla_debug_attend_mma.argtypes = [vp, i64, vp, i64, vp, i64, vp, i32, i32, i32, f32, f32, i32, i32, vp, vp,
                                         vp]
    lib.mla_plan_units.argtypes = [i32, i32, i32, vp, i32, i32, vp, i64, ctypes.POINTER(ctypes.c_int)]
    lib.mla_plan_units.restype = i64
    lib.mla_plan_units_ex.argtypes = [i32, i32, i32, vp, i32, i32, i32, vp, i64, ctypes.POINTER(ctypes.c_int)]
    lib.mla_plan_units_ex.restype = i64
    lib.mla_merge_splits.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp]
    lib.mla_value_gate.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp]
    lib.mla_merge_value_gate.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp]
    lib.mla_choose_splits.argtypes = [i32, i32, i32, i32, i64, vp, i32, ctypes.POINTER(ctypes.c_int)]
    lib.mla_debug_gather.argtypes = [vp, i64, vp, i64, vp, i32, i64, vp, vp]
    lib.mla_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint)]
    lib.mla_debug_wait_timeout.argtypes = [vp]
    lib.mla_kv_append.argtypes = [vp, i64, vp, i64, vp, i64, f32, vp, i64, vp]
    lib.mla_decode_step_static.argtypes = [vp, i64, vp, i64, vp, i64, vp, i32, i32, i32, f32, f32, i32, i32,
                                           vp, i64, vp, vp, vp, vp, vp, vp, vp]
    lib.mla_add_rms_norm.argtypes = [vp, i64, i32, vp, i64, i32, vp, f32, i64, i32, i32, f32, vp, i64, vp, vp, i64, vp]
    lib.mla_norm_rope.argtypes = [vp, i64, i64, i32, vp, i32, f32, vp, vp, i64, i32, i32, ctypes.c_uint, i64, i32, i32,
                                  i32, f32, vp, i64, vp, i64, i64, vp, vp]
    lib.mla_query_absorb.argtypes = [vp, i64, i64, vp, vp, vp, i64, ctypes.c_uint, i64, i32, f32, vp, i64, vp]
    lib.mla_index_scores.argtypes = [vp, vp, vp, vp, i64, vp, i64, vp, i32, i32, i32, f32, vp, ctypes.c_uint, vp]
    lib.mla_index_select.argtypes = [vp, vp, i64, vp, i32, i32, i32, i32, i32, i32, ctypes.c_uint, vp, i64, vp, vp]
    lib.mla_index_select_capacity.argtypes = [i32, i32, i64, i32, i32]
    lib.mla_index_select_capacity.restype = i64
    lib.mla_token_weights.argtypes = [vp, i64, vp, i64, vp, i64, vp, i32, i32, i32, f32, f32, f32, vp, f32, vp, vp,
                                      ctypes.c_uint, vp, i64, vp]
    lib.mla_token_weights_workspace.argtypes = [i32, i32, i64, ctypes.c_uint]
    lib.mla_token_weights_workspace.restype = i64
    lib.mla_kv_evict.argtypes = [vp, i64, vp, i32, vp, vp, i32, i32, i32, vp, vp, vp, vp]
    lib.mla_value_gate_lora.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, i64, vp]
    lib.mla_value_gate_lora_workspace.argtypes = [i32, i32, i32, i32]
    lib.mla_value_gate_lora_workspace.restype = i64
    for name in ("mla_norm_rope", "mla_query_absorb", "mla_index_scores", "mla_index_select", "mla_add_rms_norm", "mla_token_weights", "mla_kv_evict", "mla_value_gate_lora",
                 "mla_decode_attend", "mla_decode_attend_ex", "mla_decode_attend_paged", "mla_decode_attend_planned", "mla_merge_splits", "mla_value_gate", "mla_merge_value_gate", "mla_debug_gather",
                 "mla_device_status", "mla_choose_splits", "mla_kv_append", "mla_debug_wait_timeout",
                 "mla_decode_step_static", "mla_debug_attend_mma"):
        getattr(lib, name).restype = ctypes.c_int
    lib.mla_status_string.argtypes = [ctypes.c_int]
    lib.mla_status_string.restype = ctypes.c_char_p
    lib.mla_last_error.restype = ctypes.c_char_p
    lib.mla_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _status_name(status: int) -> str:
    try:
        return library().mla_status_string(status).decode()
    except Exception:  # pragma: no cover - only when the library is absent
        return "status"


def _check(status: int, where: str):
    if status != MLA_OK:
        raise MlaError(status, where, library().mla_last_error().decode())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device=None) -> int:
    if stream is None:
        if _raw_stream is not None:   # the current stream's handle without building a Stream object
            return int(_raw_stream(torch.cuda.current_device() if device is None else device))
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


class Prepared:
    """A validated call with its arguments marshalled once: calling it
    launches on ``stream`` (default: the current stream of the tensors'
    device) with no further checks.  The tensors it was prepared from must
    stay alive with their shapes and addresses (as for a captured CUDA
    graph); their contents may change between calls.  ``outputs`` holds what
    the plain call returns."""

    def __init__(self, fn, args, where, device, outputs, keep):
        self._fn, self._args, self._where, self._device = fn, args, where, device
        self.outputs, self._keep = outputs, keep

    def __call__(self, stream=None):
        st = self._fn(*self._args, ctypes.c_void_p(_stream(stream, self._device)))
        if st != MLA_OK:
            _check(st, self._where)
        return self.outputs


def _marshal(fn, args):
    """Arguments converted to their ctypes types once (None and ctypes
    instances as they are)."""
    return [a if a is None or isinstance(a, ctypes._SimpleCData) else t(a) for t, a in zip(fn.argtypes, args)]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def _same_device(dev, **named):
    """Every given tensor lives on the CUDA device ``dev``: a host pointer or
    another device's pointer handed to a kernel would fault."""
    _need(dev.type == "cuda", "tensors must be CUDA tensors (got %s)" % dev)
    for name, t in named.items():
        if t is not None:
            _need(t.device == dev, "%s is on %s, expected %s" % (name, t.device, dev))


def _buffer(t, name, dtype, shape):
    """A caller-supplied output: exactly this dtype and shape, contiguous
    (the kernels write every element of that extent)."""
    _need(t.dtype == dtype and tuple(t.shape) == tuple(shape) and t.is_contiguous(),
          "%s must be a contiguous %s tensor of shape %s" % (name, dtype, list(shape)))


def _as_u8(kv: torch.Tensor) -> torch.Tensor:
    if kv.dtype == torch.float8_e4m3fn:
        kv = kv.view(torch.uint8)
    _need(kv.dtype == torch.uint8, "kv must be uint8 codes or float8_e4m3fn")
    return kv


def attend(q, kv, pages, indptr, scale, kv_scale, num_splits, split_tokens, *, heads=None, qlen=1,
           o=None, lse=None, causal=False, page_size=1, last_page_len=None, q_scale=1.0, plan=None, stream=None,
           prepare=False):
    """Split-KV attention: returns ``(o [num_splits, S, heads, 512] bf16,
    lse [num_splits, S, heads] f32)``.

    ``q``: bf16 ``[S, H_pad, 576]`` whose rows may be strided (a padded query:
    ``heads`` < H_pad reads only the first ``heads``); ``kv``: ``[pool, 576]``
    fp8 codes; ``pages``/``indptr``: int32; S = (len(indptr) - 1) * qlen.
    ``causal``: row tq of a request sees only its first L - qlen + tq + 1
    tokens (``mla_decode_attend_ex`` with ``MLA_ATTEND_CAUSAL``).
    ``page_size`` > 1: block tables (``pages`` = block indices, ``indptr``
    counts blocks, ``last_page_len`` int32 [R] rows used in each request's
    last block; ``mla_decode_attend_paged``).
    A ``q`` of dtype float8_e4m3fn / uint8 is an fp8 query (codes); its
    ``q_scale`` multiplies the softmax scale (``MLA_ATTEND_Q_FP8``).
    ``plan``: a device int32 work plan from :func:`plan_units` for the same
    lengths and shape (``mla_decode_attend_planned``): its splits replace
    the ``split_tokens`` rule; the merged result is the same up to rounding.
    ``prepare=True`` validates and marshals once and returns a
    :class:`Prepared` call (launch it with ``call(stream)``) instead of
    launching.
    """
    kv = _as_u8(kv)
    heads = q.shape[1] if heads is None else heads
    R = indptr.numel() - 1
    S = R * qlen
    q8 = q.dtype in (torch.float8_e4m3fn, torch.uint8)
    if q.dtype == torch.float8_e4m3fn:
        q = q.view(torch.uint8)
    _need((q8 or q.dtype == torch.bfloat16) and q.dim() == 3 and q.shape[2] == D_QK,
          "q must be bf16 or fp8 e4m3 [S, H, 576]")
    _need(q.stride(2) == 1 and q.stride(1) == D_QK, "q rows must have contiguous [H, 576] heads")
    _need(q.shape[0] == S and heads <= q.shape[1], "q shape does not match indptr / qlen / heads")
    _need(kv.dim() == 2 and kv.shape[1] == D_QK and kv.is_contiguous(), "kv must be contiguous [pool, 576]")
    _need(pages.dtype == torch.int32 and indptr.dtype == torch.int32, "pages / indptr must be int32")
    _need(pages.is_contiguous() and indptr.is_contiguous(), "pages / indptr must be contiguous")
    _same_device(q.device, kv=kv, pages=pages, indptr=indptr, o=o, lse=lse, plan=plan,
                 last_page_len=last_page_len if page_size > 1 else None)
    if o is None:
        o = torch.empty((num_splits, S, heads, D_LATENT), dtype=torch.bfloat16, device=q.device)
    else:
        _buffer(o, "o", torch.bfloat16, (num_splits, S, heads, D_LATENT))
    if lse is None:
        lse = torch.empty((num_splits, S, heads), dtype=torch.float32, device=q.device)
    else:
        _buffer(lse, "lse", torch.float32, (num_splits, S, heads))
    if page_size > 1:
        _need(last_page_len is not None and last_page_len.dtype == torch.int32 and last_page_len.numel() == R
              and last_page_len.is_contiguous(), "page_size > 1 needs last_page_len int32 [R]")
    if plan is not None:
        _need(plan.dtype == torch.int32 and plan.dim() == 1 and plan.is_contiguous(),
              "plan must be a contiguous int32 device tensor")
    args = (_ptr(q), q.stride(0), _ptr(kv), kv.shape[0], _ptr(pages), pages.numel(), _ptr(indptr),
            _ptr(last_page_len) if page_size > 1 else None, int(page_size), R, qlen,
            heads, float(scale), float(kv_scale), float(q_scale), int(num_splits), int(split_tokens), _ptr(o),
            _ptr(lse), (ATTEND_CAUSAL if causal else 0) | (ATTEND_Q_FP8 if q8 else 0), _ptr(plan),
            0 if plan is None else plan.numel())
    lib = library()
    if prepare:
        # marshal once: ctypes converts each argument on every call otherwise
        conv = _marshal(lib.mla_decode_attend_planned, args)
        return Prepared(lib.mla_decode_attend_planned, conv, "mla_decode_attend", q.device.index, (o, lse),
                        (q, kv, pages, indptr, last_page_len, plan))
    st = lib.mla_decode_attend_planned(*args, ctypes.c_void_p(_stream(stream, q.device.index)))
    _check(st, "mla_decode_attend")
    return o, lse


def debug_attend_mma(q, kv, pages, indptr, scale, kv_scale, num_splits, split_tokens, *, heads=None, qlen=1,
                     o=None, lse=None, stream=None):
    """The same partials as :func:`attend` (page size 1, bf16 query, no
    options) from the library's second attend kernel, the warp-MMA one that
    the tests run as a cross-check (``mla_debug_attend_mma``)."""
    kv = _as_u8(kv)
    heads = q.shape[1] if heads is None else heads
    R = indptr.numel() - 1
    S = R * qlen
    _need(q.dtype == torch.bfloat16 and q.dim() == 3 and q.shape[2] == D_QK and q.stride(2) == 1
          and q.stride(1) == D_QK, "q must be bf16 [S, H, 576] with contiguous [H, 576] heads")
    _need(q.shape[0] == S and heads <= q.shape[1], "q shape does not match indptr / qlen / heads")
    _need(kv.dim() == 2 and kv.shape[1] == D_QK and kv.is_contiguous(), "kv must be contiguous [pool, 576]")
    _need(pages.dtype == torch.int32 and indptr.dtype == torch.int32 and pages.is_contiguous()
          and indptr.is_contiguous(), "pages / indptr must be contiguous int32")
    _same_device(q.device, kv=kv, pages=pages, indptr=indptr, o=o, lse=lse)
    if o is None:
        o = torch.empty((num_splits, S, heads, D_LATENT), dtype=torch.bfloat16, device=q.device)
    else:
        _buffer(o, "o", torch.bfloat16, (num_splits, S, heads, D_LATENT))
    if lse is None:
        lse = torch.empty((num_splits, S, heads), dtype=torch.float32, device=q.device)
    else:
        _buffer(lse, "lse", torch.float32, (num_splits, S, heads))
    st = library().mla_debug_attend_mma(_ptr(q), q.stride(0), _ptr(kv), kv.shape[0], _ptr(pages), pages.numel(),
                                        _ptr(indptr), R, qlen, heads, float(scale), float(kv_scale), int(num_splits),
                                        int(split_tokens), _ptr(o), _ptr(lse),
                                        ctypes.c_void_p(_stream(stream, q.device.index)))
    _check(st, "mla_debug_attend_mma")
    return o, lse


def merge(o, lse, *, latent=None, lse_out=None, want_lse=True, stream=None):
    """LSE merge: returns ``(latent [S, heads, 512] bf16, lse [S, heads] f32 or None)``."""
    _need(o.dtype == torch.bfloat16 and o.dim() == 4 and o.shape[3] == D_LATENT and o.is_contiguous(),
          "o must be contiguous bf16 [splits, S, heads, 512]")
    _need(lse.dtype == torch.float32 and lse.shape == o.shape[:3] and lse.is_contiguous(),
          "lse must be contiguous f32 [splits, S, heads]")
    ns, S, H = o.shape[:3]
    _same_device(o.device, lse=lse, latent=latent, lse_out=lse_out)
    if latent is None:
        latent = torch.empty((S, H, D_LATENT), dtype=torch.bfloat16, device=o.device)
    else:
        _buffer(latent, "latent", torch.bfloat16, (S, H, D_LATENT))
    if lse_out is None and want_lse:
        lse_out = torch.empty((S, H), dtype=torch.float32, device=o.device)
    elif lse_out is not None:
        _buffer(lse_out, "lse_out", torch.float32, (S, H))
    st = library().mla_merge_splits(_ptr(o), _ptr(lse), ns, S, H, _ptr(latent), _ptr(lse_out),
                                    ctypes.c_void_p(_stream(stream, o.device.index)))
    _check(st, "mla_merge_splits")
    return latent, lse_out


def value_gate(latent, w_uv, gate, lengths, qlen=1, *, out=None, stream=None):
    """W_UV + sigmoid gate: returns ``out [S, heads*128] bf16``."""
    _need(latent.dtype == torch.bfloat16 and latent.dim() == 3 and latent.shape[2] == D_LATENT
          and latent.is_contiguous(), "latent must be contiguous bf16 [S, heads, 512]")
    S, H = latent.shape[:2]
    _need(w_uv.dtype == torch.bfloat16 and tuple(w_uv.shape) == (H, D_V, D_LATENT) and w_uv.is_contiguous(),
          "w_uv must be contiguous bf16 [heads, 128, 512]")
    _need(gate.dtype == torch.bfloat16 and tuple(gate.shape) == (S, H * D_V) and gate.is_contiguous(),
          "gate must be contiguous bf16 [S, heads*128]")
    _need(lengths.dtype == torch.int32 and lengths.numel() * qlen == S and lengths.is_contiguous(),
          "lengths must be contiguous int32 [S / qlen]")
    _same_device(latent.device, w_uv=w_uv, gate=gate, lengths=lengths, out=out)
    if out is None:
        out = torch.empty((S, H * D_V), dtype=torch.bfloat16, device=latent.device)
    else:
        _buffer(out, "out", torch.bfloat16, (S, H * D_V))
    st = library().mla_value_gate(_ptr(latent), _ptr(w_uv), _ptr(gate), _ptr(lengths), lengths.numel(), qlen,
                                  H, _ptr(out), ctypes.c_void_p(_stream(stream, latent.device.index)))
    _check(st, "mla_value_gate")
    return out


def merge_value_gate(o, lse, w_uv, gate, lengths, qlen=1, *, out=None, latent=None, lse_out=None,
                     stream=None, prepare=False):
    """Merge + W_UV + gate in one call (one launch for small batches):
    returns ``out [S, heads*128] bf16``.  ``latent`` (allocated if not given)
    receives the merged latent, ``lse_out`` (optional) the merged LSE.
    ``prepare=True``: a :class:`Prepared` call instead (see :func:`attend`)."""
    _need(o.dtype == torch.bfloat16 and o.dim() == 4 and o.shape[3] == D_LATENT and o.is_contiguous(),
          "o must be contiguous bf16 [splits, S, heads, 512]")
    _need(lse.dtype == torch.float32 and lse.shape == o.shape[:3] and lse.is_contiguous(),
          "lse must be contiguous f32 [splits, S, heads]")
    ns, S, H = o.shape[:3]
    _need(w_uv.dtype == torch.bfloat16 and tuple(w_uv.shape) == (H, D_V, D_LATENT) and w_uv.is_contiguous(),
          "w_uv must be contiguous bf16 [heads, 128, 512]")
    _need(gate.dtype == torch.bfloat16 and tuple(gate.shape) == (S, H * D_V) and gate.is_contiguous(),
          "gate must be contiguous bf16 [S, heads*128]")
    _need(lengths.dtype == torch.int32 and lengths.numel() * qlen == S and lengths.is_contiguous(),
          "lengths must be contiguous int32 [S / qlen]")
    _same_device(o.device, lse=lse, w_uv=w_uv, gate=gate, lengths=lengths, out=out, latent=latent, lse_out=lse_out)
    if latent is not None:
        _buffer(latent, "latent", torch.bfloat16, (S, H, D_LATENT))
    if lse_out is not None:
        _buffer(lse_out, "lse_out", torch.float32, (S, H))
    if out is None:
        out = torch.empty((S, H * D_V), dtype=torch.bfloat16, device=o.device)
    else:
        _buffer(out, "out", torch.bfloat16, (S, H * D_V))
    if latent is None:
        latent = torch.empty((S, H, D_LATENT), dtype=torch.bfloat16, device=o.device)
    args = (_ptr(o), _ptr(lse), ns, _ptr(w_uv), _ptr(gate), _ptr(lengths), lengths.numel(), qlen, H, _ptr(out),
            _ptr(latent), _ptr(lse_out))
    lib = library()
    if prepare:
        conv = _marshal(lib.mla_merge_value_gate, args)
        return Prepared(lib.mla_merge_value_gate, conv, "mla_merge_value_gate", o.device.index, out,
                        (o, lse, w_uv, gate, lengths, out, latent, lse_out))
    st = lib.mla_merge_value_gate(*args, ctypes.c_void_p(_stream(stream, o.device.index)))
    _check(st, "mla_merge_value_gate")
    return out


def choose_splits(num_requests, qlen, heads, max_len=0, total_len=0, sm_count=0, lengths=None):
    """Host-side split plan: returns ``(num_splits, split_tokens)``.
    ``lengths`` (host-known per-request lengths, any int sequence or CPU
    tensor) makes the plan exact; otherwise ``max_len`` / ``total_len``
    estimate it."""
    st = ctypes.c_int(0)
    host = None
    if lengths is not None:
        host = torch.as_tensor(lengths, dtype=torch.int32, device="cpu").contiguous()
        num_requests = host.numel()
    ns = library().mla_choose_splits(int(num_requests), int(qlen), int(heads), int(max_len), int(total_len),
                                     None if host is None else ctypes.c_void_p(host.data_ptr()),
                                     int(sm_count), ctypes.byref(st))
    if ns < 1:
        _check(ns, "choose_splits")
    return int(ns), int(st.value)


def plan_units(lengths, qlen, heads, num_splits, sm_count=0, min_splits=1):
    """Balanced host work plan for :func:`attend` (``mla_plan_units_ex``):
    the requests cut into at most ``num_splits`` splits (and, where their
    tiles allow, at least ``min_splits``) so that each of ``sm_count`` CTAs
    (0: the current device's SMs) gets about the same number of tiles.
    Returns ``(plan, splits_used)``: a CPU int32 tensor (copy it to the
    device and pass it as ``attend(..., plan=)``) and the most splits any
    request got (the smallest ``num_splits`` the partial buffers need)."""
    host = torch.as_tensor(lengths, dtype=torch.int32, device="cpu").contiguous()
    lib = library()
    used = ctypes.c_int(0)
    args = (host.numel(), int(qlen), int(heads), ctypes.c_void_p(host.data_ptr()), int(min_splits),
            int(num_splits), int(sm_count))
    n = lib.mla_plan_units_ex(*args, None, 0, ctypes.byref(used))
    if n < 0:
        _check(int(n), "mla_plan_units_ex")
    plan = torch.empty(n, dtype=torch.int32)
    n2 = lib.mla_plan_units_ex(*args, ctypes.c_void_p(plan.data_ptr()), n, ctypes.byref(used))
    if n2 < 0:
        _check(int(n2), "mla_plan_units_ex")
    return plan, int(used.value)


def debug_gather(kv, pages, indptr, total_rows=None, stream=None):
    """Every request's KV rows in request order ([sum L, 576] uint8), gathered
    by the attend kernels' own row addressing."""
    kv = _as_u8(kv)
    _need(kv.dim() == 2 and kv.shape[1] == D_QK and kv.is_contiguous(), "kv must be contiguous [pool, 576]")
    _need(pages.dtype == torch.int32 and indptr.dtype == torch.int32 and pages.is_contiguous()
          and indptr.is_contiguous(), "pages / indptr must be contiguous int32")
    _same_device(kv.device, pages=pages, indptr=indptr)
    if total_rows is None:
        total_rows = int(indptr[-1].item())
    out = torch.empty((total_rows, D_QK), dtype=torch.uint8, device=kv.device)
    st = library().mla_debug_gather(_ptr(kv), kv.shape[0], _ptr(pages), pages.numel(), _ptr(indptr),
                                    indptr.numel() - 1, total_rows, _ptr(out),
                                    ctypes.c_void_p(_stream(stream, kv.device.index)))
    _check(st, "mla_debug_gather")
    return out


def kv_append(kv, kv_c, k_pe, slots, k_scale, *, stream=None):
    """Write new tokens into the fp8 cache in place: ``kv[slots[i]] =
    e4m3((kv_c[i] ++ k_pe[i]) / k_scale)`` (negative slots skipped).

    ``kv``: uint8 / float8_e4m3fn ``[pool, 576]``; ``kv_c``: bf16 ``[T, 512]``
    and ``k_pe``: bf16 ``[T, 64]`` (rows may be strided); ``slots``: int64
    ``[T]``.  Returns ``kv``.
    """
    kvu = _as_u8(kv)
    _need(kvu.dim() == 2 and kvu.shape[1] == D_QK and kvu.is_contiguous(), "kv must be contiguous [pool, 576]")
    _need(kv_c.dtype == torch.bfloat16 and kv_c.dim() == 2 and kv_c.shape[1] == D_LATENT and kv_c.stride(1) == 1,
          "kv_c must be bf16 [T, 512] with contiguous rows")
    _need(k_pe.dtype == torch.bfloat16 and k_pe.dim() == 2 and k_pe.shape[1] == D_QK - D_LATENT and k_pe.stride(1) == 1,
          "k_pe must be bf16 [T, 64] with contiguous rows")
    T = kv_c.shape[0]
    _need(k_pe.shape[0] == T and slots.dtype == torch.int64 and slots.numel() == T and slots.is_contiguous(),
          "slots must be contiguous int64 [T] matching kv_c / k_pe")
    _same_device(kvu.device, kv_c=kv_c, k_pe=k_pe, slots=slots)
    st = library().mla_kv_append(_ptr(kv_c), kv_c.stride(0), _ptr(k_pe), k_pe.stride(0), _ptr(slots), T,
                                 float(k_scale), _ptr(kvu), kvu.shape[0],
                                 ctypes.c_void_p(_stream(stream, kvu.device.index)))
    _check(st, "mla_kv_append")
    return kv


_NORM_QUANT = {None: 0, "row": 1, "group": 2, "static": 3}
_ops_module = None


def _ops():
    """The compiled Python module (``csrc/binding.cpp``) of the calls below:
    it checks the arguments (ValueError), allocates the outputs and calls the
    library with the tensors' device current, on ``stream`` or the device's
    current stream; raises if it has not been built."""
    global _ops_module
    if _ops_module is None:
        library()
        path = _build.ops_path()
        if not os.path.exists(path):
            raise RuntimeError("mla_decode_paged_gb300: native module %s is missing; run "
                               "mla_decode_paged_gb300.build() first (no fallback exists)" % path)
        loader = importlib.machinery.ExtensionFileLoader("mla_ops", path)
        spec = importlib.util.spec_from_file_location("mla_ops", path, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        _ops_module = module
    return _ops_module


def add_rms_norm(x, weight, eps, residual=None, *, quant=None, scale=None, out=None, out_scales=None,
                 residual_out=None, stream=None):
    """Residual addition and root-mean-square norm (``mla_add_rms_norm``):
    returns ``(out, out_scales, residual_out)`` (None for what does not
    apply).

    ``x``: bf16 / fp16 ``[T, D]``, rows may be strided (D a multiple of 8);
    ``weight``: x's type ``[D]``; ``residual``: x's type or float32 ``[T, D]``:
    the norm is of the float32 sum, which ``residual_out`` gets rounded to
    the residual's type (pass ``residual`` itself to update it in place).
    ``quant=None``: ``out`` in x's type.  Otherwise e4m3 codes
    (float8_e4m3fn) with scales ``"row"`` ``[T]``, ``"group"``
    ``[T, ceil(D / 128)]`` (128 columns each) or ``"static"`` (the float
    ``scale``; no scales returned): a code stands for code * scale.
    """
    q = _NORM_QUANT.get(quant)
    if q is None:
        raise ValueError("quant must be None, 'row', 'group' or 'static'")
    r = (_ops_module or _ops()).add_rms_norm(x, weight, eps, residual, q, scale, out, out_scales, residual_out, stream)
    if type(r) is int:
        _check(r, "mla_add_rms_norm")
    return r


_ROPE_QUANT = {None: 0, "head": 1, "static": 3}


def norm_rope(x, weight=None, eps=1e-6, *, positions=None, cos_sin=None, rope_start=0, interleaved=False, quant=None,
              scale=None, slots=None, out=None, out_scales=None, stream=None):
    """Norm and position rotation of every head in one pass
    (``mla_norm_rope``): returns ``(out, out_scales)`` (None for what does
    not apply).

    ``x``: bf16 / fp16 ``[T, H, D]`` or ``[T, D]`` (one head), rows and heads
    may be strided (D a multiple of 8 up to 1,024).  ``weight``: x's type
    ``[n]``: the root-mean-square norm of a head's first n columns (None: no
    norm).  ``positions``: int64 ``[T]`` and ``cos_sin``: float32
    ``[positions, d]``, d / 2 cosines then d / 2 sines: columns
    ``rope_start`` to ``rope_start + d`` are rotated after the norm, column i
    with i + d / 2, or with ``interleaved`` 2i with 2i + 1 (None: no
    rotation).  ``quant=None``: ``out`` in x's type.  Otherwise e4m3 codes
    (float8_e4m3fn) with scales ``"head"`` ``[T, H]`` or ``"static"`` (the
    float ``scale``; no scales returned): a code stands for code * scale.
    ``slots``: int64 ``[T]``: token t goes to row ``slots[t]`` of ``out``
    (and of ``out_scales``), a cache of any number of rows; negative slots
    are skipped.  ``out=x`` works in place.  Codes and scales that are both new
    share an allocation, which either of them keeps.  A static scale divides
    columns that are neither normed nor rotated as :func:`kv_append` does, to
    the same codes.
    """
    q = _ROPE_QUANT.get(quant)
    if q is None:
        raise ValueError("quant must be None, 'head' or 'static'")
    r = (_ops_module or _ops()).norm_rope(x, weight, eps, positions, cos_sin, rope_start, interleaved, q, scale, slots,
                                          out, out_scales, stream)
    if type(r) is int:
        _check(r, "mla_norm_rope")
    return r


def query_absorb(q, w_uk, *, positions=None, cos_sin=None, interleaved=False, q_scale=None, out=None, stream=None):
    """The query that :func:`attend` takes (``mla_query_absorb``): returns
    ``out [S, H, 576]``, its first 512 columns the product of a head's first
    128 with ``w_uk[h]``, its last 64 the head's last 64, rotated.

    ``q``: bf16 ``[S, H, 192]``, rows and heads may be strided (H up to 128);
    ``w_uk``: bf16 ``[H, 128, 512]``; ``positions``: int64 ``[S]`` and
    ``cos_sin``: float32 ``[positions, 64]`` as in :func:`norm_rope`, whose
    column pairs ``interleaved`` picks (None: no rotation).  ``q_scale``: the
    output is e4m3 codes that stand for code * q_scale, for
    ``attend(..., q_scale=q_scale)`` (None: bf16).  ``out``: a tensor of
    ``[S, H or more, 576]`` whose first H heads are written (a padded query).
    """
    r = (_ops_module or _ops()).query_absorb(q, w_uk, positions, cos_sin, interleaved, q_scale, out, stream)
    if type(r) is int:
        _check(r, "mla_query_absorb")
    return r


def token_weights(q, kv, pages, indptr, scale, kv_scale, lse, *, heads=None, qlen=1, weights=None, decay=1.0,
                  causal=False, q_scale=1.0, out=None, workspace=None, stream=None):
    """The attention weight every cached token received in a decode step,
    added to ``decay`` times the weights gathered so far
    (``mla_token_weights``): returns ``out`` float32 ``[len(pages)]``.

    ``q``, ``kv``, ``pages``, ``indptr``, ``scale``, ``kv_scale``, ``heads``,
    ``qlen``, ``causal``, ``q_scale`` as in :func:`attend` (page size 1);
    ``lse``: the step's merged LSE float32 ``[S, heads]`` (from
    :func:`merge` or :func:`decode_step`).  ``weights``: float32, one entry
    per entry of ``pages`` (None: zeros); ``out=weights`` updates in place.
    Entries before ``indptr[0]`` and from ``indptr[-1]`` on belong to no
    request and are left as they were (a new ``out`` holds nothing there).
    ``workspace``: uint8,
    at least :func:`token_weights_workspace` bytes, 16-byte aligned
    (allocated if not given and needed; not shared by calls that may
    overlap).
    """
    r = (_ops_module or _ops()).token_weights(q, kv, pages, indptr, scale, kv_scale, lse, heads, qlen, weights, decay,
                                              causal, q_scale, out, workspace, stream)
    if type(r) is int:
        _check(r, "mla_token_weights")
    return r


def token_weights_workspace(qlen, heads, num_pages, fp8_query=False):
    """Bytes of workspace that :func:`token_weights` needs."""
    n = library().mla_token_weights_workspace(qlen, heads, num_pages, ATTEND_Q_FP8 if fp8_query else 0)
    if n < 0:
        _check(int(n), "mla_token_weights_workspace")
    return n


def index_scores(q, weights, k, pages, indptr, *, q_scales=None, scale=1.0, qlen=1, causal=False, out=None,
                 stream=None):
    """A cheap score of every cached token for every query row
    (``mla_index_scores``): returns ``out`` float32 ``[qlen, len(pages)]``,
    ``out[tq, i] = scale * sum_h weights[t, h] * q_scales[t, h] *
    max(0, <q[t, h], k[pages[i]]>)`` for the tokens i of row t's request,
    -inf with ``causal`` where row tq does not see the token.

    ``q``: e4m3 codes (float8_e4m3fn or uint8) ``[S, H, 128]``, H up to 128,
    S = (len(indptr) - 1) * qlen; ``weights`` and ``q_scales`` (None: ones):
    float32 ``[S, H]`` (both from :func:`norm_rope` with ``quant="head"`` and
    a projection); ``k``: e4m3 codes ``[pool, 128]``, the index cache
    (:func:`norm_rope` with ``slots`` writes it; its static scale goes into
    ``scale``); ``pages`` and ``indptr`` as in :func:`attend`.  Entries that
    belong to no request are left as they were (a new ``out`` holds nothing
    there).
    """
    r = (_ops_module or _ops()).index_scores(q, weights, k, pages, indptr, q_scales, scale, qlen, causal, out, stream)
    if type(r) is int:
        _check(r, "mla_index_scores")
    return r


def index_select(scores, pages, indptr, topk, *, block=1, recent=0, sinks=0, causal=False, pages_out=None,
                 indptr_out=None, stream=None):
    """The tokens that each query row attends to (``mla_index_select``):
    returns ``(pages_out, indptr_out)``, a page list a query row.

    ``scores``: float32 ``[qlen, len(pages)]`` from :func:`index_scores`;
    ``pages`` / ``indptr``: the requests' lists.  A row's tokens (with
    ``causal`` those it sees) in blocks of ``block`` (a power of two up to
    256): its last ``recent`` blocks, its first ``sinks`` and, between them,
    those of largest maximal score, ``topk`` blocks in all (equal ones by the
    lower position); ``recent`` is at least 1 with ``block`` > 1.
    ``indptr_out`` int32 ``[R * qlen + 1]`` and ``pages_out`` (at least
    :func:`index_select_capacity` entries, -1 behind the last list) go to
    :func:`attend` with ``qlen=1``: every query row a request of its own,
    whose length, min(tokens, topk * block) for blocks of one token, does not
    depend on the scores.  Two new outputs share an allocation, which either
    of them keeps (the indptr alone the whole page list's).
    """
    r = (_ops_module or _ops()).index_select(scores, pages, indptr, topk, block, recent, sinks, causal, pages_out,
                                             indptr_out, stream)
    if type(r) is int:
        _check(r, "mla_index_select")
    return r


def index_select_capacity(requests, qlen, num_pages, topk, block=1):
    """Entries of ``pages_out`` that :func:`index_select` needs."""
    n = library().mla_index_select_capacity(requests, qlen, num_pages, topk, block)
    if n < 0:
        _check(int(n), "mla_index_select_capacity")
    return n


def kv_evict(pages, indptr, weights, budget, *, recent=0, sinks=0, pages_out=None, indptr_out=None, weights_out=None,
             stream=None):
    """Cut every request's page list to ``budget`` tokens (``mla_kv_evict``):
    its last ``recent``, its first ``sinks`` and, between them, the heaviest
    by ``weights`` (float32, one per entry of ``pages``; from
    :func:`token_weights`).  Returns ``(pages_out, indptr_out,
    weights_out)``: ``pages_out`` holds the kept rows of every request in
    order (``indptr_out`` counts them; both go to :func:`attend` as they
    are), then the freed rows, ``indptr[-1] - indptr[0]`` rows in all (what
    lies behind them in a longer list's outputs is not written);
    ``weights_out`` the kept tokens' weights, then zeros, likewise.  At most
    65,536 requests.  A row that several requests hold (a shared prefix) may be
    kept by one and freed by another.  ``budget``: an int, or int32 ``[R]``
    on the device.
    """
    r = (_ops_module or _ops()).kv_evict(pages, indptr, weights, budget, recent, sinks, pages_out, indptr_out,
                                         weights_out, stream)
    if type(r) is int:
        _check(r, "mla_kv_evict")
    return r


def value_gate_lora(latent, w_uv, gate, lengths, lora_a, lora_b, adapters, lora_scale, qlen=1, *, out=None,
                    workspace=None, stream=None):
    """:func:`value_gate` with one low-rank adapter per request beside W_UV
    (``mla_value_gate_lora``): returns ``out [S, heads*128] bf16``.

    ``lora_a``: bf16 ``[n, rank, 512]``, ``lora_b``: bf16 ``[n, heads*128,
    rank]`` (rank a multiple of 8 up to 128), ``lora_scale``: float32
    ``[n]``; ``adapters``: int32 ``[R]``, request r's adapter, -1 for none.
    ``workspace``: uint8, at least :func:`value_gate_lora_workspace` bytes,
    16-byte aligned (allocated if not given; not shared by calls that may
    overlap).
    """
    r = (_ops_module or _ops()).value_gate_lora(latent, w_uv, gate, lengths, lora_a, lora_b, adapters, lora_scale, qlen,
                                                out, workspace, stream)
    if type(r) is int:
        _check(r, "mla_value_gate_lora")
    return r


def value_gate_lora_workspace(requests, qlen, heads, rank):
    """Bytes of workspace that :func:`value_gate_lora` needs."""
    n = library().mla_value_gate_lora_workspace(requests, qlen, heads, rank)
    if n < 0:
        _check(int(n), "mla_value_gate_lora_workspace")
    return n


def debug_wait_timeout(stream=None):
    """Test hook: enqueue a kernel whose bounded wait runs out (about 2 s);
    it sets DEV_TIMEOUT, which :func:`device_status` then reports."""
    _check(library().mla_debug_wait_timeout(ctypes.c_void_p(_stream(stream))), "mla_debug_wait_timeout")


def device_status(stream=None) -> int:
    """Synchronise the stream, return and clear the device status bits
    (DEV_BAD_PAGE, DEV_BAD_INDPTR, DEV_TIMEOUT, DEV_BAD_PLAN,
    DEV_BAD_ADAPTER, DEV_BAD_POSITION)."""
    flags = ctypes.c_uint(0)
    _check(library().mla_device_status(ctypes.c_void_p(_stream(stream)), ctypes.byref(flags)),
           "mla_device_status")
    return int(flags.value)


def decode_step(q, kv, pages, indptr, scale, kv_scale, w_uv, gate, lengths, *, heads=None, qlen=1,
                num_splits=None, split_tokens=None, max_len=None, total_len=0, causal=False, page_size=1,
                last_page_len=None, q_scale=1.0, plan=None, stream=None):
    """The whole step (attend, then the merge with value/gate through
    :func:`merge_value_gate`: one launch for small batches); returns
    ``(out, latent, lse)``.  Without a split plan one is chosen from
    ``max_len`` (host-known longest request).  ``causal``, ``page_size``,
    ``last_page_len``, ``q_scale`` and ``plan`` as in :func:`attend`."""
    heads = q.shape[1] if heads is None else heads
    if num_splits is None or split_tokens is None:
        if max_len is None:
            raise ValueError("give num_splits and split_tokens, or max_len for the split plan")
        num_splits, split_tokens = choose_splits(indptr.numel() - 1, qlen, heads, max_len, total_len)
    o, lse = attend(q, kv, pages, indptr, scale, kv_scale, num_splits, split_tokens, heads=heads,
                    qlen=qlen, causal=causal, page_size=page_size, last_page_len=last_page_len,
                    q_scale=q_scale, plan=plan, stream=stream)
    lse_m = torch.empty(lse.shape[1:], dtype=torch.float32, device=lse.device)
    latent = torch.empty(o.shape[1:], dtype=torch.bfloat16, device=o.device)
    out = merge_value_gate(o, lse, w_uv, gate, lengths, qlen, latent=latent, lse_out=lse_m, stream=stream)
    return out, latent, lse_m


def decode_step_static(q, kv, pages, indptr, scale, kv_scale, w_uv, gate, lengths, num_splits, split_tokens, *,
                       heads=None, qlen=1, plan=None, out=None, latent=None, lse_out=None, stream=None):
    """The whole step through ``mla_decode_step_static``: the split partials
    live in the library's own 32 MiB device buffer, so the native call
    allocates nothing (for callers that cannot allocate device memory while
    they run; see the header).  Returns ``(out, latent, lse_out)``; the
    outputs are allocated here with torch unless given.  Calls on one
    device share the buffer: keep them ordered on one stream.  The first
    call on a device looks up the buffer's address, so make it before any
    stream capture.  Raises :class:`MlaError` (MLA_ERR_UNSUPPORTED) when the
    partials, ``num_splits * S * heads * 1028`` bytes, do not fit."""
    kv = _as_u8(kv)
    heads = q.shape[1] if heads is None else heads
    R = indptr.numel() - 1
    S = R * qlen
    _need(q.dtype == torch.bfloat16 and q.dim() == 3 and q.shape[2] == D_QK and q.stride(2) == 1
          and q.stride(1) == D_QK, "q must be bf16 [S, H, 576] with contiguous [H, 576] heads")
    _need(q.shape[0] == S and heads <= q.shape[1], "q shape does not match indptr / qlen / heads")
    _need(kv.dim() == 2 and kv.shape[1] == D_QK and kv.is_contiguous(), "kv must be contiguous [pool, 576]")
    _need(pages.dtype == torch.int32 and indptr.dtype == torch.int32 and pages.is_contiguous()
          and indptr.is_contiguous(), "pages / indptr must be contiguous int32")
    _need(w_uv.dtype == torch.bfloat16 and tuple(w_uv.shape) == (heads, D_V, D_LATENT) and w_uv.is_contiguous(),
          "w_uv must be contiguous bf16 [heads, 128, 512]")
    _need(gate.dtype == torch.bfloat16 and tuple(gate.shape) == (S, heads * D_V) and gate.is_contiguous(),
          "gate must be contiguous bf16 [S, heads*128]")
    _need(lengths.dtype == torch.int32 and lengths.numel() == R and lengths.is_contiguous(),
          "lengths must be contiguous int32 [R]")
    if plan is not None:
        _need(plan.dtype == torch.int32 and plan.dim() == 1 and plan.is_contiguous(),
              "plan must be a contiguous int32 device tensor")
    _same_device(q.device, kv=kv, pages=pages, indptr=indptr, w_uv=w_uv, gate=gate, lengths=lengths, plan=plan,
                 out=out, latent=latent, lse_out=lse_out)
    if out is None:
        out = torch.empty((S, heads * D_V), dtype=torch.bfloat16, device=q.device)
    else:
        _buffer(out, "out", torch.bfloat16, (S, heads * D_V))
    if latent is None:
        latent = torch.empty((S, heads, D_LATENT), dtype=torch.bfloat16, device=q.device)
    else:
        _buffer(latent, "latent", torch.bfloat16, (S, heads, D_LATENT))
    if lse_out is not None:
        _buffer(lse_out, "lse_out", torch.float32, (S, heads))
    st = library().mla_decode_step_static(
        _ptr(q), q.stride(0), _ptr(kv), kv.shape[0], _ptr(pages), pages.numel(), _ptr(indptr), R, qlen, heads,
        float(scale), float(kv_scale), int(num_splits), int(split_tokens), _ptr(plan),
        0 if plan is None else plan.numel(), _ptr(w_uv), _ptr(gate), _ptr(lengths), _ptr(out), _ptr(latent),
        _ptr(lse_out), ctypes.c_void_p(_stream(stream, q.device.index)))
    _check(st, "mla_decode_step_static")
    return out, latent, lse_out
