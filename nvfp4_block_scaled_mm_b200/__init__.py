"""NVFP4 block-scaled GEMM with a fused BF16 LoRA correction on B200 (sm_100a).

Thin ctypes binding over the C ABI in ``include/nvfp4lora.h`` (``libnvfp4lora.so``, built
in-tree by :mod:`nvfp4_block_scaled_mm_b200.build`).  It only marshals arguments: every
step of the operation runs in the library's CUDA kernels.  PyTorch supplies device
memory, the current stream and the tensors' version counters (used for the stale-adapter
check).  There is no CPU fallback: the library is loaded on first use, and a missing
library raises ``RuntimeError`` there.

Two layers:

* ``nvfp4lora_mm``, ``nvfp4lora_prepare``, ``nvfp4lora_refold``,
  ``nvfp4lora_mm_prepared`` -- one-to-one with the C entry points (torch tensors in, the
  status mapped to exceptions);
* ``mm_nvfp4_lora``, ``prepare_nvfp4_lora_adapter``, ``PreparedNvFp4LoraAdapter``,
  ``StaleAdapterError`` -- the API of flashinfer.gemm.mm_nvfp4_lora and
  flashinfer.gemm.prepare_nvfp4_lora_adapter (signatures, Parameters, Returns, Notes);
  ``grouped_mm_nvfp4_lora`` (grouped_mm_bf16's grouped form), ``fp4_quantize``, and
  ``bgmv_moe_gemm2_lora_delta`` / ``fill_w_ptr`` (flashinfer.fused_moe.bgmv_moe_gemm2_lora_delta);
* ``moe_permute`` / ``moe_unpermute`` (the grouped call's rows and tables, and back, with gradients),
  ``add_rmsnorm_fp8_quantize``, ``fp8_quantize`` and ``mm_fp8`` (the 8-bit layers beside the NVFP4 ones).
"""

from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnvfp4lora.so")

__all__ = [
    "StaleAdapterError", "PreparedNvFp4LoraAdapter", "mm_nvfp4_lora", "prepare_nvfp4_lora_adapter",
    "nvfp4lora_mm", "nvfp4lora_prepare", "nvfp4lora_refold", "nvfp4lora_mm_prepared",
    "nvfp4lora_device_status", "nvfp4lora_quantize", "fp4_quantize", "library_path", "version",
    "nvfp4lora_grouped_mm", "grouped_mm_nvfp4_lora", "nvfp4lora_bgmv_moe_gemm2_lora_delta",
    "bgmv_moe_gemm2_lora_delta", "fill_w_ptr",
    "MoePermutation", "moe_capacity", "moe_permute", "moe_permute_backward", "moe_unpermute", "moe_unpermute_backward",
    "fp8_quantize", "add_rmsnorm_fp8_quantize", "mm_fp8",
    "nvfp4lora_moe_permute", "nvfp4lora_moe_permute_backward", "nvfp4lora_moe_unpermute",
    "nvfp4lora_moe_unpermute_backward", "nvfp4lora_fp8_quantize", "nvfp4lora_rmsnorm_fp8_quantize", "nvfp4lora_mm_fp8",
]

OK, INVALID_ARG, STALE, ALPHA_ZERO, UNSUPPORTED_ARCH, DEVICE_TIMEOUT, CUDA_ERR = range(7)


class StaleAdapterError(RuntimeError):
    """A prepared adapter's alpha, lora_b or lora_scale changed since its last (re)fold."""


class DeviceTimeoutError(RuntimeError):
    """A kernel's bounded wait ran out (reported by :func:`nvfp4lora_device_status`)."""


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m nvfp4_block_scaled_mm_b200.build` "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, U64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_int32
    lib.nvfp4lora_mm.argtypes = [P, P, P, I64, P, I64, P, P, P, P, I64, P, P, I64, I64, I64, P]
    lib.nvfp4lora_mm.restype = ctypes.c_int
    lib.nvfp4lora_prepare.argtypes = [P, P, P, I64, I64, P, P, U64, P, P]
    lib.nvfp4lora_prepare.restype = ctypes.c_int
    lib.nvfp4lora_refold.argtypes = [P, P, P, P, I64, I64, U64, P]
    lib.nvfp4lora_refold.restype = ctypes.c_int
    lib.nvfp4lora_mm_prepared.argtypes = [P, P, P, I64, P, I64, P, P, P, P, P, U64, P, P, I64, I64, I64, P]
    lib.nvfp4lora_mm_prepared.restype = ctypes.c_int
    lib.nvfp4lora_device_status.argtypes = [P]
    lib.nvfp4lora_device_status.restype = ctypes.c_int
    lib.nvfp4lora_selftest_wait_timeout.argtypes = [I64, P]
    lib.nvfp4lora_selftest_wait_timeout.restype = ctypes.c_int
    lib.nvfp4lora_quantize.argtypes = [P, I64, I64, P, P, P, I64, P]
    lib.nvfp4lora_quantize.restype = ctypes.c_int
    lib.nvfp4lora_grouped_mm.argtypes = [P, P, P, I64, P, I64, P, I64, P, P, P, P, I64, P, P, I64, I64, I64, P]
    lib.nvfp4lora_grouped_mm.restype = ctypes.c_int
    lib.nvfp4lora_bgmv_moe_gemm2_lora_delta.argtypes = [P, I64, I64, P, P, I64, P, I64, P, P, P, I64, I64, I64, I64,
                                                        I64, ctypes.c_int32, ctypes.c_float, ctypes.c_int32, P, P]
    lib.nvfp4lora_bgmv_moe_gemm2_lora_delta.restype = ctypes.c_int
    lib.nvfp4lora_moe_permute.argtypes = [P, I64, I64, P, I64, I64, I64, I32, P, I64, P, P, P, P, I64, P]
    lib.nvfp4lora_moe_permute.restype = ctypes.c_int
    lib.nvfp4lora_moe_unpermute.argtypes = [P, I64, I64, I32, P, P, I64, I64, P, P]
    lib.nvfp4lora_moe_unpermute.restype = ctypes.c_int
    lib.nvfp4lora_moe_permute_backward.argtypes = [P, I64, I64, I32, P, I64, I64, P, P]
    lib.nvfp4lora_moe_permute_backward.restype = ctypes.c_int
    lib.nvfp4lora_moe_unpermute_backward.argtypes = [P, P, I64, I64, I32, P, P, P, I64, P, I64, I64, P, P, P]
    lib.nvfp4lora_moe_unpermute_backward.restype = ctypes.c_int
    lib.nvfp4lora_fp8_quantize.argtypes = [P, I64, I64, I32, I64, P, P, I64, I64, P]
    lib.nvfp4lora_fp8_quantize.restype = ctypes.c_int
    lib.nvfp4lora_rmsnorm_fp8_quantize.argtypes = [P, P, P, I64, I64, I32, ctypes.c_float, P, P, P, I64, I64, P]
    lib.nvfp4lora_rmsnorm_fp8_quantize.restype = ctypes.c_int
    lib.nvfp4lora_mm_fp8.argtypes = [P, P, P, I64, I64, P, P, P, I32, I64, I64, I64, P]
    lib.nvfp4lora_mm_fp8.restype = ctypes.c_int
    lib.nvfp4lora_last_error.argtypes = []
    lib.nvfp4lora_last_error.restype = ctypes.c_char_p
    lib.nvfp4lora_version.argtypes = []
    lib.nvfp4lora_version.restype = ctypes.c_char_p
    return lib


class _LazyLib:
    """Loads libnvfp4lora.so on first attribute access (raises if it was never built)."""

    _handle = None

    def __getattr__(self, name):
        if _LazyLib._handle is None:
            _LazyLib._handle = _load()
        value = getattr(_LazyLib._handle, name)
        self.__dict__[name] = value
        return value


_lib = _LazyLib()


def library_path() -> str:
    return LIB_PATH


def load_library():
    """Load the CUDA library now (it is otherwise loaded on first use)."""
    _lib.nvfp4lora_version  # noqa: B018
    return LIB_PATH


def version() -> str:
    return _lib.nvfp4lora_version().decode()


class _Adapter(ctypes.Structure):
    _fields_ = [("b_folded", ctypes.c_void_p), ("ratio", ctypes.c_void_p), ("alpha", ctypes.c_void_p),
                ("lora_b", ctypes.c_void_p), ("lora_scale", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("r", ctypes.c_int64), ("src_version", ctypes.c_uint64), ("device", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def _check(status: int) -> None:
    if status == OK:
        return
    msg = _lib.nvfp4lora_last_error().decode()
    if status in (INVALID_ARG, ALPHA_ZERO):
        raise ValueError(msg)
    if status == STALE:
        raise StaleAdapterError(msg)
    if status == DEVICE_TIMEOUT:
        raise DeviceTimeoutError(msg)
    raise RuntimeError(msg)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _launch(fn, anchor: torch.Tensor, stream, *args) -> None:
    """Run a C entry point on `stream`, or on the current stream of the anchor tensor's device, with the stream's
    device current (the library launches on the current device)."""
    if stream is None:
        _call(fn, anchor.device, *args)
    else:
        with torch.cuda.device(stream.device):
            _check(fn(*args, stream.cuda_stream))


def _written(*tensors) -> None:
    """Count a write by address in the version counters of the caller's buffers (None: not given), as an in-place
    operation of torch does: autograd then refuses to use a saved tensor that a call has overwritten."""
    given = [t for t in tensors if t is not None]
    if given:
        increment_version(given)


def _version_token(lora_b: torch.Tensor, lora_scale: torch.Tensor) -> int:
    return ((lora_b._version & 0xFFFFFFFF) << 32) | (lora_scale._version & 0xFFFFFFFF)


# --------------------------------------------------------------------------------------
# one-to-one C ABI wrappers
# --------------------------------------------------------------------------------------

def nvfp4lora_mm(a, b, a_sf, b_sf, alpha, d, lora_b, lora_scale, r, bias, out, M, N, K, stream=None):
    _check(_lib.nvfp4lora_mm(_ptr(a), _ptr(b), _ptr(a_sf), a_sf.numel(), _ptr(b_sf), b_sf.numel(),
                             _ptr(alpha), _ptr(d), _ptr(lora_b), _ptr(lora_scale), int(r), _ptr(bias),
                             _ptr(out), int(M), int(N), int(K), _stream(stream)))
    _written(out)
    return out


def nvfp4lora_prepare(lora_b, lora_scale, alpha, N, r, b_folded, ratio, src_version, stream=None):
    adp = _Adapter()
    _check(_lib.nvfp4lora_prepare(_ptr(lora_b), _ptr(lora_scale), _ptr(alpha), int(N), int(r),
                                  _ptr(b_folded), _ptr(ratio), int(src_version), ctypes.byref(adp),
                                  _stream(stream)))
    return adp


def nvfp4lora_refold(adp, lora_b, lora_scale, alpha, N, r, src_version, stream=None):
    _check(_lib.nvfp4lora_refold(ctypes.byref(adp), _ptr(lora_b), _ptr(lora_scale), _ptr(alpha),
                                 int(N), int(r), int(src_version), _stream(stream)))
    return adp


def nvfp4lora_mm_prepared(a, b, a_sf, b_sf, alpha, d, adp, cur_lora_b, cur_lora_scale, cur_version,
                          bias, out, M, N, K, stream=None):
    _check(_lib.nvfp4lora_mm_prepared(_ptr(a), _ptr(b), _ptr(a_sf), a_sf.numel(), _ptr(b_sf),
                                      b_sf.numel(), _ptr(alpha), _ptr(d), ctypes.byref(adp),
                                      _ptr(cur_lora_b), _ptr(cur_lora_scale), int(cur_version),
                                      _ptr(bias), _ptr(out), int(M), int(N), int(K), _stream(stream)))
    _written(out)
    return out


def nvfp4lora_grouped_mm(a, b, a_sf, b_sf, m_indptr, num_experts, alpha, d, lora_b, lora_scale, r, bias, out,
                         rows, N, K, stream=None):
    _check(_lib.nvfp4lora_grouped_mm(_ptr(a), _ptr(b), _ptr(a_sf), a_sf.numel(), _ptr(b_sf), b_sf.numel(),
                                     _ptr(m_indptr), int(num_experts), _ptr(alpha), _ptr(d), _ptr(lora_b),
                                     _ptr(lora_scale), int(r), _ptr(bias), _ptr(out), int(rows), int(N), int(K),
                                     _stream(stream)))
    _written(out)
    return out


def nvfp4lora_bgmv_moe_gemm2_lora_delta(act, padded_rows, I, perm, w_ptr_a, lora_stride_a, w_ptr_b, lora_stride_b,
                                        topk_ids, topk_weights, lora_ids, num_tokens, top_k, num_experts, rank,
                                        hidden_size, lora_dtype, scale, out_dtype, out, stream=None):
    _check(_lib.nvfp4lora_bgmv_moe_gemm2_lora_delta(
        _ptr(act), int(padded_rows), int(I), _ptr(perm), _ptr(w_ptr_a), int(lora_stride_a), _ptr(w_ptr_b),
        int(lora_stride_b), _ptr(topk_ids), _ptr(topk_weights), _ptr(lora_ids), int(num_tokens), int(top_k),
        int(num_experts), int(rank), int(hidden_size), int(lora_dtype), float(scale), int(out_dtype), _ptr(out),
        _stream(stream)))
    _written(out)
    return out


def nvfp4lora_moe_permute(x, num_tokens, row_bytes, topk_ids, top_k, num_experts, align, zero_padding, rows,
                          padded_rows, m_indptr, expanded_idx_to_permuted_idx, permuted_idx_to_expanded_idx,
                          workspace=None, workspace_bytes=0, stream=None):
    _launch(_lib.nvfp4lora_moe_permute, m_indptr, stream, _ptr(x), int(num_tokens), int(row_bytes), _ptr(topk_ids),
            int(top_k), int(num_experts), int(align), int(bool(zero_padding)), _ptr(rows), int(padded_rows),
            _ptr(m_indptr), _ptr(expanded_idx_to_permuted_idx), _ptr(permuted_idx_to_expanded_idx), _ptr(workspace),
            int(workspace_bytes))
    _written(rows, m_indptr, expanded_idx_to_permuted_idx, permuted_idx_to_expanded_idx, workspace)
    return rows


def nvfp4lora_moe_unpermute(y, padded_rows, H, dtype, expanded_idx_to_permuted_idx, topk_weights, num_tokens, top_k,
                            out, stream=None):
    _launch(_lib.nvfp4lora_moe_unpermute, out, stream, _ptr(y), int(padded_rows), int(H), int(dtype),
            _ptr(expanded_idx_to_permuted_idx), _ptr(topk_weights), int(num_tokens), int(top_k), _ptr(out))
    _written(out)
    return out


def nvfp4lora_moe_permute_backward(grad_rows, padded_rows, H, dtype, expanded_idx_to_permuted_idx, num_tokens, top_k,
                                   grad_x, stream=None):
    _launch(_lib.nvfp4lora_moe_permute_backward, grad_x, stream, _ptr(grad_rows), int(padded_rows), int(H), int(dtype),
            _ptr(expanded_idx_to_permuted_idx), int(num_tokens), int(top_k), _ptr(grad_x))
    _written(grad_x)
    return grad_x


def nvfp4lora_moe_unpermute_backward(grad_out, y, padded_rows, H, dtype, expanded_idx_to_permuted_idx,
                                     permuted_idx_to_expanded_idx, m_indptr, num_experts, topk_weights, num_tokens,
                                     top_k, grad_rows, grad_weights, stream=None):
    _launch(_lib.nvfp4lora_moe_unpermute_backward, m_indptr, stream, _ptr(grad_out), _ptr(y), int(padded_rows), int(H),
            int(dtype), _ptr(expanded_idx_to_permuted_idx), _ptr(permuted_idx_to_expanded_idx), _ptr(m_indptr),
            int(num_experts), _ptr(topk_weights), int(num_tokens), int(top_k), _ptr(grad_rows), _ptr(grad_weights))
    _written(grad_rows, grad_weights)
    return grad_rows, grad_weights


def nvfp4lora_fp8_quantize(x, rows, H, dtype, block_rows, q, scales, scale_stride_row, scale_stride_group, stream=None):
    _launch(_lib.nvfp4lora_fp8_quantize, q, stream, _ptr(x), int(rows), int(H), int(dtype), int(block_rows), _ptr(q),
            _ptr(scales), int(scale_stride_row), int(scale_stride_group))
    _written(q, scales)
    return q, scales


def nvfp4lora_rmsnorm_fp8_quantize(x, residual, weight, rows, H, dtype, eps, norm_out, q, scales, scale_stride_row,
                                   scale_stride_group, stream=None):
    _launch(_lib.nvfp4lora_rmsnorm_fp8_quantize, q, stream, _ptr(x), _ptr(residual), _ptr(weight), int(rows), int(H),
            int(dtype), float(eps), _ptr(norm_out), _ptr(q), _ptr(scales), int(scale_stride_row),
            int(scale_stride_group))
    _written(residual, norm_out, q, scales)
    return q, scales


def nvfp4lora_mm_fp8(a, b, a_scale, a_scale_stride_m, a_scale_stride_k, b_scale, bias, out, out_dtype, M, N, K,
                     stream=None):
    _launch(_lib.nvfp4lora_mm_fp8, out, stream, _ptr(a), _ptr(b), _ptr(a_scale), int(a_scale_stride_m),
            int(a_scale_stride_k), _ptr(b_scale), _ptr(bias), _ptr(out), int(out_dtype), int(M), int(N), int(K))
    _written(out)
    return out


def nvfp4lora_device_status(stream=None) -> None:
    """Synchronise the stream; raise DeviceTimeoutError if a kernel's wait ran out, ValueError if a
    table read on the device (a grouped call's m_indptr, a LoRA delta's or a permutation's routing) broke its rules."""
    _check(_lib.nvfp4lora_device_status(_stream(stream)))


def nvfp4lora_quantize(x, rows, K, global_scale, codes, scales, stream=None):
    _check(_lib.nvfp4lora_quantize(_ptr(x), int(rows), int(K), _ptr(global_scale), _ptr(codes), _ptr(scales),
                                   scales.numel(), _stream(stream)))
    _written(codes, scales)
    return codes, scales


def nvfp4lora_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    """Enqueue the bounded-wait self-test: a wait that nothing completes runs out after
    limit_ns; the next nvfp4lora_device_status raises DeviceTimeoutError."""
    _check(_lib.nvfp4lora_selftest_wait_timeout(int(limit_ns), _stream(stream)))


# --------------------------------------------------------------------------------------
# the pages' API
# --------------------------------------------------------------------------------------

def _need(t, name, dtype, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")


def _same_device(anchor_name: str, anchor: torch.Tensor, **others) -> None:
    """Every tensor given must live on the anchor tensor's device: the kernels run on that device
    and read every operand by address there, so an operand on another GPU would be read through
    a foreign address.  ValueError names the first tensor that differs (None entries are
    skipped)."""
    device = anchor.device
    for name, t in others.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device} but {anchor_name} is on {anchor.device}: "
                             "every tensor of a call must be on the same device")


class PreparedNvFp4LoraAdapter:
    """A folded adapter (prepare_nvfp4_lora_adapter, Returns): ``b_folded`` bf16 [N, r], the
    device ``ratio`` scalar, the alpha tensor it belongs to, and the pins of its sources."""

    def __init__(self, c_adapter: _Adapter, b_folded, ratio, alpha, lora_b, lora_scale):
        self._c = c_adapter
        self.b_folded = b_folded
        self.ratio = ratio
        self.alpha = alpha
        self.lora_b = lora_b
        self.lora_scale = lora_scale

    @property
    def N(self) -> int:
        return int(self._c.N)

    @property
    def r(self) -> int:
        return int(self._c.r)


def _check_fold_inputs(lora_b, lora_scale, alpha):
    _need(lora_b, "lora_b", torch.bfloat16, 2)
    _need(lora_scale, "lora_scale", torch.float32)
    _need(alpha, "alpha", torch.float32)
    if lora_scale.numel() != 1:
        raise ValueError("lora_scale must be a one-element fp32 tensor")
    if alpha.numel() < 1:
        raise ValueError("alpha must hold at least one element")


def prepare_nvfp4_lora_adapter(lora_b: torch.Tensor, lora_scale: torch.Tensor, alpha: torch.Tensor, *,
                               out: Optional[PreparedNvFp4LoraAdapter] = None) -> PreparedNvFp4LoraAdapter:
    """Fold ``b_folded = bf16(lora_b * (lora_scale / alpha[0]))``.

    ``out=None``: the eager form (one host read of (lora_scale, alpha); alpha == 0 or a
    non-finite ratio raises ValueError).  ``out=adapter``: in-place refold on the device,
    no host read, graph-capturable; alpha must be the adapter's own alpha tensor.
    """
    _check_fold_inputs(lora_b, lora_scale, alpha)
    _same_device("lora_b", lora_b, lora_scale=lora_scale, alpha=alpha,
                 b_folded=None if out is None else out.b_folded, ratio=None if out is None else out.ratio)
    N, r = lora_b.shape
    stream = torch.cuda.current_stream(lora_b.device)
    if out is None:
        with torch.cuda.device(lora_b.device):
            b_folded = torch.empty_like(lora_b)
            ratio = torch.empty(1, dtype=torch.float32, device=lora_b.device)
            c = nvfp4lora_prepare(lora_b, lora_scale, alpha, N, r, b_folded, ratio,
                                  _version_token(lora_b, lora_scale), stream)
        return PreparedNvFp4LoraAdapter(c, b_folded, ratio, alpha, lora_b, lora_scale)
    if not isinstance(out, PreparedNvFp4LoraAdapter):
        raise ValueError("out must be a PreparedNvFp4LoraAdapter")
    with torch.cuda.device(lora_b.device):
        nvfp4lora_refold(out._c, lora_b, lora_scale, alpha, N, r, _version_token(lora_b, lora_scale), stream)
    out.lora_b = lora_b
    out.lora_scale = lora_scale
    return out


def mm_nvfp4_lora(a: torch.Tensor, b: torch.Tensor, a_sf: torch.Tensor, b_sf: torch.Tensor,
                  alpha: torch.Tensor, d: Optional[torch.Tensor] = None,
                  lora_b: Optional[torch.Tensor] = None, lora_scale: Optional[torch.Tensor] = None, *,
                  lora_adapter: Optional[PreparedNvFp4LoraAdapter] = None,
                  bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  out_dtype: torch.dtype = torch.bfloat16, backend: str = "cake",
                  enable_pdl: Optional[bool] = None) -> torch.Tensor:
    """``out = alpha * (dequant(a) @ dequant(b)^T) + lora_scale * (d @ lora_b^T) [+ bias]``.

    Raw path: ``d``, ``lora_b``, ``lora_scale``; ``lora_scale=None`` is the adapter-off
    call even if d / lora_b are given.  Prepared path: ``lora_adapter=`` plus ``d``.

    The call returns once the kernel is enqueued.  A kernel whose bounded wait gives up (a
    stalled pipeline) returns early and leaves ``out`` partly unwritten, so ``out`` is defined
    only once a later :func:`nvfp4lora_device_status` on the stream has returned without
    raising ``DeviceTimeoutError``.
    """
    if out_dtype != torch.bfloat16:
        raise ValueError("out_dtype: only torch.bfloat16 is supported")
    if backend not in ("cake", "auto"):
        raise ValueError("backend must be 'cake' or 'auto'")
    if enable_pdl not in (None, True):
        raise ValueError("enable_pdl must be None or True")
    if lora_adapter is not None and (lora_b is not None or lora_scale is not None):
        raise ValueError("pass either the raw adapter (lora_b, lora_scale) or lora_adapter, not both")
    _need(a, "a", torch.uint8, 2)
    _need(b, "b", torch.uint8, 2)
    _need(a_sf, "a_sf", torch.uint8)
    _need(b_sf, "b_sf", torch.uint8)
    _need(alpha, "alpha", torch.float32)
    M, K = a.shape[0], a.shape[1] * 2
    N = b.shape[0]
    if b.shape[1] * 2 != K:
        raise ValueError(f"a is [M, K/2] = {tuple(a.shape)} but b is {tuple(b.shape)}: K differs")
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, 1)
        if bias.shape[0] != N:
            raise ValueError(f"bias must be [N] = [{N}]")
    _same_device("a", a, b=b, a_sf=a_sf, b_sf=b_sf, alpha=alpha, d=d, lora_b=lora_b, lora_scale=lora_scale,
                 bias=bias, out=out,
                 b_folded=None if lora_adapter is None else lora_adapter.b_folded,
                 ratio=None if lora_adapter is None else lora_adapter.ratio)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    else:
        _need(out, "out", torch.bfloat16, 2)
        if tuple(out.shape) != (M, N):
            raise ValueError(f"out must be [M, N] = [{M}, {N}]")
    stream = torch.cuda.current_stream(a.device)
    with torch.cuda.device(a.device):
        if lora_adapter is not None:
            if d is None:
                raise ValueError("the prepared path still requires d")
            _need(d, "d", torch.bfloat16, 2)
            if tuple(d.shape) != (M, lora_adapter.r):
                raise ValueError(f"d must be [M, r] = [{M}, {lora_adapter.r}]")
            src = lora_adapter
            nvfp4lora_mm_prepared(a, b, a_sf, b_sf, alpha, d, src._c, src.lora_b, src.lora_scale,
                                  _version_token(src.lora_b, src.lora_scale), bias, out, M, N, K, stream)
            return out
        if lora_scale is None:
            nvfp4lora_mm(a, b, a_sf, b_sf, alpha, None, None, None, 0, bias, out, M, N, K, stream)
            return out
        _need(lora_scale, "lora_scale", torch.float32)
        if lora_scale.numel() != 1:
            raise ValueError("lora_scale must be a one-element fp32 tensor")
        if d is None or lora_b is None:
            raise ValueError("the raw path needs d and lora_b with lora_scale")
        _need(d, "d", torch.bfloat16, 2)
        _need(lora_b, "lora_b", torch.bfloat16, 2)
        r = d.shape[1]
        if d.shape[0] != M or tuple(lora_b.shape) != (N, r):
            raise ValueError(f"d must be [M, r] and lora_b [N, r]; got {tuple(d.shape)}, {tuple(lora_b.shape)}")
        nvfp4lora_mm(a, b, a_sf, b_sf, alpha, d, lora_b, lora_scale, r, bias, out, M, N, K, stream)
        return out


def grouped_mm_nvfp4_lora(a: torch.Tensor, b: torch.Tensor, a_sf: torch.Tensor, b_sf: torch.Tensor,
                          m_indptr: torch.Tensor, alpha: torch.Tensor, d: Optional[torch.Tensor] = None,
                          lora_b: Optional[torch.Tensor] = None, lora_scale: Optional[torch.Tensor] = None, *,
                          bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Grouped (expert-partitioned) form, flashinfer.grouped_mm.grouped_mm_bf16's formula applied to
    :func:`mm_nvfp4_lora`: for each expert e with rows ``s, t = m_indptr[e], m_indptr[e+1]``,
    ``out[s:t] = alpha[e] * (dequant(a[s:t]) @ dequant(b[e])^T) + lora_scale * (d[s:t] @ lora_b[e]^T)
    [+ bias[e]]``.

    a: uint8 [rows, K/2] with a_sf over all rows; b: uint8 [E, N, K/2] with b_sf holding E
    consecutive 128x4 buffers; m_indptr: int32 [E + 1] on the device, 0, non-decreasing multiples
    of 128, at most rows (each expert's rows fill whole 128-row scale blocks); alpha: fp32 [E];
    d: bf16 [rows, r]; lora_b: bf16 [E, N, r]; lora_scale: fp32 [1] or None; bias: bf16 [E, N].
    Rows from m_indptr[E] on are left untouched.  m_indptr is checked on the device: a table that
    breaks its rules computes nothing, and :func:`nvfp4lora_device_status` raises ValueError.
    """
    _need(a, "a", torch.uint8, 2)
    _need(b, "b", torch.uint8, 3)
    _need(a_sf, "a_sf", torch.uint8)
    _need(b_sf, "b_sf", torch.uint8)
    _need(m_indptr, "m_indptr", torch.int32, 1)
    _need(alpha, "alpha", torch.float32, 1)
    rows, K = a.shape[0], a.shape[1] * 2
    E, N = b.shape[0], b.shape[1]
    if b.shape[2] * 2 != K:
        raise ValueError(f"a is [rows, K/2] = {tuple(a.shape)} but b is {tuple(b.shape)}: K differs")
    if m_indptr.shape[0] != E + 1 or alpha.shape[0] != E:
        raise ValueError(f"m_indptr must be [E + 1] = [{E + 1}] and alpha [E] = [{E}]")
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, 2)
        if tuple(bias.shape) != (E, N):
            raise ValueError(f"bias must be [E, N] = [{E}, {N}]")
    r = 0
    if lora_scale is not None:
        _need(lora_scale, "lora_scale", torch.float32)
        if lora_scale.numel() != 1:
            raise ValueError("lora_scale must be a one-element fp32 tensor")
        if d is None or lora_b is None:
            raise ValueError("the LoRA term needs d and lora_b with lora_scale")
        _need(d, "d", torch.bfloat16, 2)
        _need(lora_b, "lora_b", torch.bfloat16, 3)
        r = d.shape[1]
        if d.shape[0] != rows or tuple(lora_b.shape) != (E, N, r):
            raise ValueError(f"d must be [rows, r] and lora_b [E, N, r]; got {tuple(d.shape)}, {tuple(lora_b.shape)}")
    if out is None:
        out = torch.empty((rows, N), dtype=torch.bfloat16, device=a.device)
    else:
        _need(out, "out", torch.bfloat16, 2)
        if tuple(out.shape) != (rows, N):
            raise ValueError(f"out must be [rows, N] = [{rows}, {N}]")
    _same_device("a", a, b=b, a_sf=a_sf, b_sf=b_sf, m_indptr=m_indptr, alpha=alpha, d=d, lora_b=lora_b,
                 lora_scale=lora_scale, bias=bias, out=out)
    with torch.cuda.device(a.device):
        nvfp4lora_grouped_mm(a, b, a_sf, b_sf, m_indptr, E, alpha, d if lora_scale is not None else None,
                             lora_b if lora_scale is not None else None, lora_scale, r, bias, out, rows, N, K,
                             torch.cuda.current_stream(a.device))
    return out


_DTYPE_CODES = {torch.bfloat16: 0, torch.float16: 1}


def fill_w_ptr(banks) -> torch.Tensor:
    """The int64 ``[1, num_experts]`` table of bank addresses that
    :func:`bgmv_moe_gemm2_lora_delta` takes as ``w_ptr_a`` / ``w_ptr_b``: entry e is the device
    address of ``banks[e]`` (one contiguous bf16 or fp16 CUDA tensor per expert, holding that
    expert's adapters ``lora_stride`` elements apart).  The table does not keep the banks alive."""
    banks = list(banks)
    if not banks:
        raise ValueError("fill_w_ptr needs at least one bank")
    dev = banks[0].device
    for i, t in enumerate(banks):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"bank {i} must be a contiguous CUDA tensor")
        if t.dtype not in _DTYPE_CODES:
            raise ValueError(f"bank {i} must be bf16 or fp16, got {t.dtype}")
        if t.device != dev:
            raise ValueError(f"bank {i} is on {t.device} but bank 0 is on {dev}")
    return torch.tensor([[t.data_ptr() for t in banks]], dtype=torch.int64, device=dev)


def bgmv_moe_gemm2_lora_delta(gemm1_activation_output: torch.Tensor, expanded_idx_to_permuted_idx: torch.Tensor,
                              w_ptr_a: torch.Tensor, lora_stride_a: int, w_ptr_b: torch.Tensor,
                              lora_stride_b: int, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                              lora_ids: torch.Tensor, rank: int, hidden_size: int, *,
                              lora_dtype: torch.dtype = torch.bfloat16, scale: float = 1.0,
                              out_dtype: torch.dtype = torch.bfloat16,
                              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """FC2 (down projection) LoRA delta of a routed MoE, flashinfer.fused_moe.bgmv_moe_gemm2_lora_delta:
    ``delta[t] = scale * sum_j topk_weights[t, j] * (B_down[l, e] @ (A_down[l, e] @ act[p]))`` with
    ``l = lora_ids[t]`` (negative: a zero row), ``e = topk_ids[t, j]`` and
    ``p = expanded_idx_to_permuted_idx[t * top_k + j]`` (negative: inactive slot).  Returns
    ``[T, hidden_size]`` in out_dtype, to be added to the MoE output.

    gemm1_activation_output: lora_dtype ``[padded_rows, I]`` (I % 8 == 0); the index, id and weight
    tensors are int32 / int32 / fp32 as shaped on the page; ``w_ptr_a`` / ``w_ptr_b``: int64
    ``[1, num_experts]`` bank-address tables (:func:`fill_w_ptr`), A_down[l, e] being the
    ``[rank, I]`` row-major block ``l * lora_stride_a`` elements into expert e's A bank and
    B_down[l, e] the ``[H, rank]`` block ``l * lora_stride_b`` elements into its B bank.  The banks
    must live on the activation's device; adapter ids must exist in them.  Routing entries are
    read on the device: one out of range is skipped and :func:`nvfp4lora_device_status` raises
    ValueError."""
    act = gemm1_activation_output
    if lora_dtype not in _DTYPE_CODES or out_dtype not in _DTYPE_CODES:
        raise ValueError("lora_dtype and out_dtype must be torch.bfloat16 or torch.float16")
    _need(act, "gemm1_activation_output", lora_dtype, 2)
    _need(expanded_idx_to_permuted_idx, "expanded_idx_to_permuted_idx", torch.int32)
    _need(w_ptr_a, "w_ptr_a", torch.int64)
    _need(w_ptr_b, "w_ptr_b", torch.int64)
    _need(topk_ids, "topk_ids", torch.int32, 2)
    _need(topk_weights, "topk_weights", torch.float32, 2)
    _need(lora_ids, "lora_ids", torch.int32, 1)
    T, top_k = topk_ids.shape
    E = w_ptr_a.numel()
    if w_ptr_b.numel() != E:
        raise ValueError(f"w_ptr_a has {E} entries but w_ptr_b has {w_ptr_b.numel()}")
    if tuple(topk_weights.shape) != (T, top_k) or lora_ids.shape[0] != T:
        raise ValueError(f"topk_weights must be [T, top_k] = [{T}, {top_k}] and lora_ids [T]")
    if expanded_idx_to_permuted_idx.numel() != T * top_k:
        raise ValueError(f"expanded_idx_to_permuted_idx must hold T * top_k = {T * top_k} entries")
    H = int(hidden_size)
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=act.device)
    else:
        _need(out, "out", out_dtype, 2)
        if tuple(out.shape) != (T, H):
            raise ValueError(f"out must be [T, hidden_size] = [{T}, {H}]")
    _same_device("gemm1_activation_output", act, expanded_idx_to_permuted_idx=expanded_idx_to_permuted_idx,
                 w_ptr_a=w_ptr_a, w_ptr_b=w_ptr_b, topk_ids=topk_ids, topk_weights=topk_weights, lora_ids=lora_ids,
                 out=out)
    with torch.cuda.device(act.device):
        nvfp4lora_bgmv_moe_gemm2_lora_delta(act, act.shape[0], act.shape[1], expanded_idx_to_permuted_idx, w_ptr_a,
                                            lora_stride_a, w_ptr_b, lora_stride_b, topk_ids, topk_weights, lora_ids,
                                            T, top_k, E, rank, H, _DTYPE_CODES[lora_dtype], scale,
                                            _DTYPE_CODES[out_dtype], out, torch.cuda.current_stream(act.device))
    return out


def fp4_quantize(x: torch.Tensor, global_scale: torch.Tensor, *, codes: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None):
    """Quantize bf16 ``x [rows, K]`` into the operand format of :func:`mm_nvfp4_lora`: E2M1
    ``codes uint8 [rows, K/2]`` and UE4M3 ``scales`` (16 K-elements each, 128x4 swizzled, rows
    padded to 128), with the per-tensor ``global_scale`` (fp32, one element, on the device) folded
    in: ``value(code) * value(scale) / global_scale`` approximates x.  Rule (per 16-block, fp32):
    ``scale = e4m3(amax * gs / 6)``, ``code = e2m1(x * gs / value(scale))``, round to nearest
    even, saturating."""
    _need(x, "x", torch.bfloat16, 2)
    _need(global_scale, "global_scale", torch.float32)
    if global_scale.numel() != 1:
        raise ValueError("global_scale must be a one-element fp32 tensor")
    _same_device("x", x, global_scale=global_scale, codes=codes, scales=scales)
    rows, K = x.shape
    if K % 64 != 0:
        raise ValueError(f"K = {K}: a multiple of 64 is required")
    nbytes = (rows + 127) // 128 * 128 * (K // 16)
    if codes is None:
        codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=x.device)
    else:
        _need(codes, "codes", torch.uint8, 2)
        if tuple(codes.shape) != (rows, K // 2):
            raise ValueError(f"codes must be [rows, K/2] = [{rows}, {K // 2}]")
    if scales is None:
        scales = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    else:
        _need(scales, "scales", torch.uint8)
    with torch.cuda.device(x.device):
        nvfp4lora_quantize(x, rows, K, global_scale, codes, scales, torch.cuda.current_stream(x.device))
    return codes, scales

# --------------------------------------------------------------------------------------
# routed tokens: rows sorted by expert for the grouped call, and back
# --------------------------------------------------------------------------------------

_ROW_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_SELF_COUNT_SLOTS = 4096      # more slots than this take a workspace
_COUNT_CHUNKS = 64


# The current stream's handle without building a Stream object (2.3 us less per call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, device: torch.device, *args) -> None:
    """Run a C entry point on the current stream of the tensors' device (the last argument it takes)."""
    index = device.index
    if torch.cuda.current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != OK:
        _check(status)


class MoePermutation(NamedTuple):
    """Routed tokens sorted by expert (:func:`moe_permute`): ``rows [capacity, H]``, ``m_indptr``
    int32 ``[E + 1]`` (the grouped call's), ``expanded_idx_to_permuted_idx`` int32 ``[T, top_k]``
    (the LoRA delta's; -1 for an inactive slot) and ``permuted_idx_to_expanded_idx`` int32
    ``[capacity]`` (-1 for rows of no slot)."""

    rows: torch.Tensor
    m_indptr: torch.Tensor
    expanded_idx_to_permuted_idx: torch.Tensor
    permuted_idx_to_expanded_idx: torch.Tensor


def moe_capacity(num_tokens: int, top_k: int, num_experts: int, align: int = 128) -> int:
    """The rows that any routing of ``num_tokens`` tokens to ``top_k`` of ``num_experts`` experts can
    need with segments of multiples of ``align`` rows."""
    n = num_tokens * top_k
    return (n + min(num_experts, n) * (align - 1)) // align * align


def _need_row_dtype(t, name):
    if not isinstance(t, torch.Tensor) or t.dtype not in _ROW_DTYPES:
        raise ValueError(f"{name} must be a torch.bfloat16, torch.float16 or torch.float32 tensor")


def _moe_permute(x, topk_ids, num_experts, align, zero_padding, out):
    T, top_k = topk_ids.shape
    capacity = out.shape[0]
    n = T * top_k
    m_indptr = topk_ids.new_empty(num_experts + 1)
    idx = torch.empty_like(topk_ids)
    inv = topk_ids.new_empty(capacity)
    work = topk_ids.new_empty(_COUNT_CHUNKS * num_experts) if n > _SELF_COUNT_SLOTS else None
    _call(_lib.nvfp4lora_moe_permute, x.device, x.data_ptr(), T, x.shape[1] * x.element_size(), topk_ids.data_ptr(),
          top_k, num_experts, align, 1 if zero_padding else 0, out.data_ptr(), capacity, m_indptr.data_ptr(),
          idx.data_ptr(), inv.data_ptr(), None if work is None else work.data_ptr(),
          0 if work is None else 4 * work.numel())
    return out, m_indptr, idx, inv


def _refuse_recording_in_capture(name: str, instead: str) -> None:
    # The gradient's accumulation nodes of leaves that an eager graph keeps alive belong to the stream
    # they were made on: running them inside a capture on another stream breaks the capture, and the
    # process ends with it.
    if torch.cuda.is_current_stream_capturing():
        raise ValueError(f"{name} of tensors that require gradients does not record a graph while a CUDA graph is being "
                         f"captured: call it on detached tensors and capture {instead}")


def _refuse_gradient_in_capture(name: str) -> None:
    if torch.cuda.is_current_stream_capturing():
        raise ValueError(f"the recorded gradient of {name} does not run while a CUDA graph is being captured: call "
                         f"{name}_backward inside the capture")


def _refuse_gradients(call: str, names: str, *tensors) -> None:
    """A call that records no graph refuses tensors that ask for one (None: not given): its results would lose their
    gradients without an error.  Under torch.no_grad() nothing is asked for.  `names`: the tensors', for the message."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                key = next(k for k, u in zip(names.split(), tensors) if u is t)
                raise ValueError(f"{call} records no gradient and {key} requires one: detach it, or call under torch.no_grad()")
    if forward_ad._current_level >= 0:
        _refuse_tangents(call, names, *tensors)


def _plain_operands(call: str, anchor_name: str, anchor: torch.Tensor, **others) -> None:
    """:func:`_same_device` and :func:`_refuse_gradients` of a call's tensors, in one pass over them."""
    device, asks = anchor.device, torch.is_grad_enabled()
    if asks and anchor.requires_grad:
        _refuse_gradients(call, anchor_name, anchor)
    for name, t in others.items():
        if t is not None:
            if t.device != device:
                _same_device(anchor_name, anchor, **{name: t})
            if asks and t.requires_grad:
                _refuse_gradients(call, name, t)
    if forward_ad._current_level >= 0:
        _refuse_tangents(call, " ".join((anchor_name, *others)), anchor, *others.values())


def _refuse_tangents(call: str, names: str, *tensors) -> None:
    """Inside a forward-mode context (forward_ad._current_level >= 0)."""
    for key, t in zip(names.split(), tensors):
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise ValueError(f"{call} has no forward-mode derivative and {key} carries a tangent")


class _MoePermuteFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, topk_ids, num_experts, align, zero_padding, capacity):
        rows, m_indptr, idx, inv = _moe_permute(x, topk_ids, num_experts, align, zero_padding,
                                                x.new_empty((capacity, x.shape[1])))
        ctx.save_for_backward(idx)
        ctx.mark_non_differentiable(m_indptr, idx, inv)
        return rows, m_indptr, idx, inv

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_rows, *_):
        _refuse_gradient_in_capture("moe_permute")
        (idx,) = ctx.saved_tensors
        return moe_permute_backward(grad_rows.contiguous(), idx), None, None, None, None, None


def moe_permute(x: torch.Tensor, topk_ids: torch.Tensor, num_experts: int, *, align: int = 128,
                zero_padding: bool = True, out: Optional[torch.Tensor] = None) -> MoePermutation:
    """Sort the rows of routed tokens by expert, for :func:`grouped_mm_nvfp4_lora` (``m_indptr``) and
    :func:`bgmv_moe_gemm2_lora_delta` (``expanded_idx_to_permuted_idx``).

    x: ``[T, H]`` of any element type, contiguous; topk_ids: int32 ``[T, top_k]`` (negative: an
    inactive slot; an expert may occur twice).  Expert e's segment holds the rows of its slots in slot
    order (``t * top_k + j``) and is padded to a multiple of ``align`` rows (128 for the grouped
    call).  Padding rows are zeros, or left as they were with ``zero_padding=False``; rows from
    ``m_indptr[E]`` on are left as they were (uninitialised without ``out``).  ``out``: a
    ``[capacity, H]`` buffer for the rows with ``capacity >= moe_capacity(T, top_k, E, align)``; it must not
    overlap x or topk_ids.  1 <= top_k <= 16, 1 <= E <= 1024.

    Differentiable in x (bf16, fp16, fp32): the gradient is :func:`moe_permute_backward`; padding
    rows' gradients are not read.  Tensors that require gradients, and a recorded gradient's own pass, are
    refused while a CUDA graph is captured (capture the two functions on detached tensors instead), and so are
    forward-mode tangents.  An id >= num_experts is read
    on the device: it counts as inactive and :func:`nvfp4lora_device_status` raises ValueError.
    """
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA tensor of 2 dimensions")
    _need(topk_ids, "topk_ids", torch.int32, 2)
    T, top_k = topk_ids.shape
    E, align = int(num_experts), int(align)
    if x.shape[0] != T:
        raise ValueError(f"x has {x.shape[0]} rows but topk_ids {T}")
    if x.shape[1] < 1:
        raise ValueError("x must have at least one column")
    if not 1 <= E <= 1024 or not 1 <= align <= 4096:
        raise ValueError(f"num_experts = {E}, align = {align}: 1 <= num_experts <= 1024 and 1 <= align <= 4096 are required")
    capacity = moe_capacity(T, top_k, E, align)
    _same_device("x", x, topk_ids=topk_ids, out=out)
    if forward_ad._current_level >= 0:
        _refuse_tangents("moe_permute", "x", x)
    if x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out is not supported for an x that requires gradients")
        _need_row_dtype(x, "x that requires gradients")
        _refuse_recording_in_capture("moe_permute", "moe_permute_backward")
        return MoePermutation(*_MoePermuteFn.apply(x, topk_ids, E, align, zero_padding, capacity))
    given = out
    if out is None:
        out = x.new_empty((capacity, x.shape[1]))
    else:
        _need(out, "out", x.dtype, 2)
        if out.shape[0] < capacity or out.shape[1] != x.shape[1]:
            raise ValueError(f"out must be [capacity, H] with capacity >= {capacity} and H = {x.shape[1]}, got {tuple(out.shape)}")
        _refuse_gradients("moe_permute into a given buffer", "out", out)
    permutation = MoePermutation(*_moe_permute(x, topk_ids, E, align, zero_padding, out))
    if given is not None:
        increment_version(given)
    return permutation


def moe_permute_backward(grad_rows: torch.Tensor, expanded_idx_to_permuted_idx: torch.Tensor, *,
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of :func:`moe_permute` by x: ``grad_x[t] = sum_j grad_rows[idx[t, j]]`` over the active
    slots, in fp32 in slot order, rounded once.  Not differentiable itself."""
    if isinstance(grad_rows, torch.Tensor):
        _refuse_gradients("moe_permute_backward", "grad_rows", grad_rows)
    return _moe_unpermute(grad_rows, expanded_idx_to_permuted_idx, None, out, "grad_rows")


def _moe_unpermute(y, idx, topk_weights, out, name="y"):
    _need_row_dtype(y, name)
    _need(y, name, y.dtype, 2)
    _need(idx, "expanded_idx_to_permuted_idx", torch.int32, 2)
    given = out
    T, top_k = idx.shape
    H = y.shape[1]
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, 2)
        if topk_weights.shape != idx.shape:
            raise ValueError(f"topk_weights must be [T, top_k] = {tuple(idx.shape)}, got {tuple(topk_weights.shape)}")
    if out is None:
        out = y.new_empty((T, H))
    else:
        _need(out, "out", y.dtype, 2)
        if out.shape != (T, H):
            raise ValueError(f"out must be [T, H] = [{T}, {H}], got {tuple(out.shape)}")
        _refuse_gradients("a sum into a given buffer", "out", out)
    _same_device(name, y, expanded_idx_to_permuted_idx=idx, topk_weights=topk_weights, out=out)
    _call(_lib.nvfp4lora_moe_unpermute, y.device, y.data_ptr(), y.shape[0], H, _ROW_DTYPES[y.dtype], idx.data_ptr(),
          None if topk_weights is None else topk_weights.data_ptr(), T, top_k, out.data_ptr())
    if given is not None:
        increment_version(given)
    return out


class _MoeUnpermuteFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, topk_weights, m_indptr, idx, inv):
        ctx.weighted = topk_weights is not None
        ctx.save_for_backward(y, topk_weights, m_indptr, idx, inv)
        return _moe_unpermute(y, idx, topk_weights, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        _refuse_gradient_in_capture("moe_unpermute")
        y, w, m_indptr, idx, inv = ctx.saved_tensors
        # rows behind the last segment get no gradient: their memory is written by no kernel
        grad_rows = torch.zeros_like(y)
        gy, gw = moe_unpermute_backward(grad_out.contiguous(), y, idx, inv, m_indptr, w, grad_rows=grad_rows)
        return gy, gw, None, None, None


def moe_unpermute(y: torch.Tensor, permutation, topk_weights: Optional[torch.Tensor] = None, *,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Bring the experts' rows back to their tokens: ``out[t] = sum_j topk_weights[t, j] * y[idx[t, j]]``
    over the token's active slots (zero without one), in fp32 in slot order, rounded once to y's type.

    y: bf16, fp16 or fp32 ``[rows, H]``; permutation: a :class:`MoePermutation`, or its
    ``expanded_idx_to_permuted_idx`` (int32 ``[T, top_k]``) alone; topk_weights: fp32 ``[T, top_k]``,
    None for weights of 1; out must not overlap an input.  An index >= rows is read on the device: it is left
    out and :func:`nvfp4lora_device_status` raises ValueError.

    Differentiable in y and topk_weights where the whole MoePermutation is given (its gradient,
    :func:`moe_unpermute_backward`, needs the tables); as for :func:`moe_permute`, not while a CUDA
    graph is captured and not in forward mode.
    """
    if forward_ad._current_level >= 0 and isinstance(y, torch.Tensor):
        _refuse_tangents("moe_unpermute", "y topk_weights", y, topk_weights)
    whole = isinstance(permutation, MoePermutation)
    idx = permutation.expanded_idx_to_permuted_idx if whole else permutation
    if torch.is_grad_enabled() and (getattr(y, "requires_grad", False) or getattr(topk_weights, "requires_grad", False)):
        if not whole:
            raise ValueError("y or topk_weights requires gradients: pass the MoePermutation, whose tables the gradient needs")
        if out is not None:
            raise ValueError("out is not supported for inputs that require gradients")
        if permutation.permuted_idx_to_expanded_idx.shape[0] != y.shape[0]:
            raise ValueError(f"y has {y.shape[0]} rows but the permutation {permutation.permuted_idx_to_expanded_idx.shape[0]}")
        _refuse_recording_in_capture("moe_unpermute", "moe_unpermute_backward")
        return _MoeUnpermuteFn.apply(y, topk_weights, permutation.m_indptr, idx, permutation.permuted_idx_to_expanded_idx)
    return _moe_unpermute(y, idx, topk_weights, out)


def moe_unpermute_backward(grad_out: torch.Tensor, y: Optional[torch.Tensor], expanded_idx_to_permuted_idx: torch.Tensor,
                           permuted_idx_to_expanded_idx: torch.Tensor, m_indptr: torch.Tensor,
                           topk_weights: Optional[torch.Tensor] = None, *, grad_rows: Optional[torch.Tensor] = None):
    """Gradients of :func:`moe_unpermute`: ``(grad_rows, grad_weights)`` with
    ``grad_rows[idx[t, j]] = topk_weights[t, j] * grad_out[t]`` and ``grad_weights[t, j] = <grad_out[t],
    y[idx[t, j]]>`` (fp32; 0 for an inactive slot; None without weights, where y is not read and may be
    None).  Padding rows of the segments get zeros; rows from ``m_indptr[E]`` on are left as they were
    in ``grad_rows`` (a ``[rows, H]`` buffer, which may be y itself and must not overlap an input otherwise;
    uninitialised there when None).  The tables are those of one :class:`MoePermutation`.  Not differentiable
    itself."""
    _need_row_dtype(grad_out, "grad_out")
    _need(grad_out, "grad_out", grad_out.dtype, 2)
    idx, inv = expanded_idx_to_permuted_idx, permuted_idx_to_expanded_idx
    _need(idx, "expanded_idx_to_permuted_idx", torch.int32, 2)
    _need(inv, "permuted_idx_to_expanded_idx", torch.int32, 1)
    _need(m_indptr, "m_indptr", torch.int32, 1)
    T, top_k = idx.shape
    rows, H = inv.shape[0], grad_out.shape[1]
    given = grad_rows
    if grad_out.shape[0] != T:
        raise ValueError(f"grad_out has {grad_out.shape[0]} rows but expanded_idx_to_permuted_idx {T}")
    grad_weights = None
    if topk_weights is not None:
        _need(topk_weights, "topk_weights", torch.float32, 2)
        if topk_weights.shape != idx.shape:
            raise ValueError(f"topk_weights must be [T, top_k] = {tuple(idx.shape)}, got {tuple(topk_weights.shape)}")
        _need(y, "y", grad_out.dtype, 2)
        if y.shape != (rows, H):
            raise ValueError(f"y must be [rows, H] = [{rows}, {H}], got {tuple(y.shape)}")
        grad_weights = torch.empty((T, top_k), dtype=torch.float32, device=grad_out.device)
    if grad_rows is None:
        grad_rows = torch.empty((rows, H), dtype=grad_out.dtype, device=grad_out.device)
    else:
        _need(grad_rows, "grad_rows", grad_out.dtype, 2)
        if grad_rows.shape != (rows, H):
            raise ValueError(f"grad_rows must be [rows, H] = [{rows}, {H}], got {tuple(grad_rows.shape)}")
    _refuse_gradients("moe_unpermute_backward", "grad_out grad_rows", grad_out, given)
    if forward_ad._current_level >= 0:
        _refuse_tangents("moe_unpermute_backward", "y topk_weights", y, topk_weights)
    _same_device("grad_out", grad_out, y=y, expanded_idx_to_permuted_idx=idx, permuted_idx_to_expanded_idx=inv,
                 m_indptr=m_indptr, topk_weights=topk_weights, grad_rows=grad_rows)
    _call(_lib.nvfp4lora_moe_unpermute_backward, grad_out.device, grad_out.data_ptr(),
          None if topk_weights is None else y.data_ptr(), rows, H, _ROW_DTYPES[grad_out.dtype], idx.data_ptr(),
          inv.data_ptr(), m_indptr.data_ptr(), m_indptr.shape[0] - 1, _ptr(topk_weights), T, top_k,
          grad_rows.data_ptr(), _ptr(grad_weights))
    if given is not None:
        increment_version(given)
    return grad_rows, grad_weights


# --------------------------------------------------------------------------------------
# 8-bit operands and product
# --------------------------------------------------------------------------------------

def _fp8_outputs(x, block_rows, q, scales):
    rows, H = x.shape
    shape = (-(-rows // block_rows), -(-H // 128))
    if q is None:
        q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    else:
        _need(q, "q", torch.float8_e4m3fn, 2)
        if q.shape != (rows, H):
            raise ValueError(f"q must be [rows, H] = [{rows}, {H}], got {tuple(q.shape)}")
    if scales is None:
        # activations' scales column-major: the product reads consecutive rows' scales together
        strides = (1, shape[0]) if block_rows == 1 else (shape[1], 1)
        scales = x.new_empty_strided(shape, strides, dtype=torch.float32)
    elif (not isinstance(scales, torch.Tensor) or scales.dtype != torch.float32 or not scales.is_cuda
          or scales.shape != shape):
        raise ValueError(f"scales must be a float32 CUDA tensor of shape {shape}")
    return q, scales


def fp8_quantize(x: torch.Tensor, *, block_rows: int = 1, q: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None):
    """Quantize ``x [rows, H]`` (bf16, fp16 or fp32) into the operand format of :func:`mm_fp8`:
    ``q`` float8_e4m3fn ``[rows, H]`` and fp32 ``scales [ceil(rows / block_rows), ceil(H / 128)]``,
    ``value(q) * scale`` approximating x.  ``block_rows=1``: a scale per 128 values of a row
    (activations; scales are column-major unless given).  ``block_rows=128``: a scale per 128 x 128
    block (weights).  Rule, in fp32: ``amax = max(max |x|, 2^-100)``, ``scale = amax / 448``,
    ``q = e4m3(x * (448 / amax))``, nearest even.  Finite values are expected: a NaN stays a NaN, an
    infinity makes its group's scale infinite, itself a NaN and the group's finite values zeros.  q and scales must not overlap x or each other.  Not differentiable: a tensor
    that requires gradients is refused outside ``torch.no_grad()``."""
    _need_row_dtype(x, "x")
    _need(x, "x", x.dtype, 2)
    if block_rows not in (1, 128):
        raise ValueError(f"block_rows = {block_rows}: 1 or 128 is required")
    given = (q, scales) if q is not None or scales is not None else None
    q, scales = _fp8_outputs(x, block_rows, q, scales)
    _plain_operands("fp8_quantize", "x", x, q=q, scales=scales)
    rows, H = x.shape
    sr, sg = scales.stride()
    _call(_lib.nvfp4lora_fp8_quantize, x.device, x.data_ptr(), rows, H, _ROW_DTYPES[x.dtype], block_rows, q.data_ptr(),
          scales.data_ptr(), sr, sg)
    if given is not None:
        _written(*given)
    return q, scales


def add_rmsnorm_fp8_quantize(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *,
                             eps: float = 1e-6, norm_out: Optional[torch.Tensor] = None,
                             q: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None):
    """Residual addition, root-mean-square norm and 8-bit quantization in one pass over ``x [rows, H]``,
    in fp32: ``h = x + residual`` (``residual`` is updated in place with the rounded h),
    ``y = h * rsqrt(mean(h^2) + eps) * weight``; returns ``(q, scales)`` of y as :func:`fp8_quantize`
    with ``block_rows=1`` gives them (from the unrounded y), the ``a`` and ``a_scale`` of
    :func:`mm_fp8`.  ``norm_out [rows, H]`` also receives y in x's type (a router or a LoRA down
    projection reads it); x may be norm_out or residual itself, and no other result overlaps another buffer of
    the call.  A row whose mean square passes fp32's range (an infinity, values of about 1e19) gives zeros, and
    NaN for its infinities.  x, weight ``[H]``, residual and norm_out share one type (bf16, fp16 or fp32).  Not differentiable: a tensor that
    requires gradients is refused outside ``torch.no_grad()``."""
    _need_row_dtype(x, "x")
    _need(x, "x", x.dtype, 2)
    H = x.shape[1]
    _need(weight, "weight", x.dtype, 1)
    if weight.shape[0] != H:
        raise ValueError(f"weight must be [H] = [{H}], got {tuple(weight.shape)}")
    for name, t in (("residual", residual), ("norm_out", norm_out)):
        if t is not None:
            _need(t, name, x.dtype, 2)
            if t.shape != x.shape:
                raise ValueError(f"{name} must be [rows, H] = {tuple(x.shape)}, got {tuple(t.shape)}")
    given = [t for t in (residual, norm_out, q, scales) if t is not None]
    q, scales = _fp8_outputs(x, 1, q, scales)
    _plain_operands("add_rmsnorm_fp8_quantize", "x", x, weight=weight, residual=residual, norm_out=norm_out, q=q, scales=scales)
    sr, sg = scales.stride()
    _call(_lib.nvfp4lora_rmsnorm_fp8_quantize, x.device, x.data_ptr(), _ptr(residual), weight.data_ptr(), x.shape[0], H,
          _ROW_DTYPES[x.dtype], eps, _ptr(norm_out), q.data_ptr(), scales.data_ptr(), sr, sg)
    if given:
        increment_version(given)
    return q, scales


def mm_fp8(a: torch.Tensor, b: torch.Tensor, a_scale: torch.Tensor, b_scale: torch.Tensor, *,
           bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
           out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """``out[m, n] = sum_kb a_scale[m, kb] * b_scale[n // 128, kb] * (a[m, kb block] . b[n, kb block]) [+ bias[n]]``
    with K blocks of 128, sums in fp32, rounded once to ``out_dtype`` (bf16, fp16 or fp32).

    a: float8_e4m3fn ``[M, K]``; b: float8_e4m3fn ``[N, K]``; a_scale: fp32 ``[M, ceil(K / 128)]`` of any
    strides (column-major, as :func:`fp8_quantize` makes it, is read fastest); b_scale: fp32
    ``[ceil(N / 128), ceil(K / 128)]`` contiguous; bias: bf16 ``[N]``; out overlaps none of them.  K % 16 == 0; any M, N >= 1.  A
    repeated call gives the same bits; the order in which a row's K blocks are added depends on the shape and on the row's
    place, so equal rows in different places may differ by the rounding of their fp32 sums.  As for
    :func:`mm_nvfp4_lora`, out is defined once a later :func:`nvfp4lora_device_status` has returned
    without raising ``DeviceTimeoutError``.  Not differentiable: a tensor that requires gradients is refused
    outside ``torch.no_grad()``."""
    _need(a, "a", torch.float8_e4m3fn, 2)
    _need(b, "b", torch.float8_e4m3fn, 2)
    _need(b_scale, "b_scale", torch.float32, 2)
    M, K = a.shape
    N = b.shape[0]
    G = -(-K // 128)
    if b.shape[1] != K:
        raise ValueError(f"a is [M, K] = {tuple(a.shape)} but b is {tuple(b.shape)}: K differs")
    if not isinstance(a_scale, torch.Tensor) or a_scale.dtype != torch.float32 or not a_scale.is_cuda:
        raise ValueError("a_scale must be a float32 CUDA tensor")
    if a_scale.shape != (M, G):
        raise ValueError(f"a_scale must be [M, ceil(K / 128)] = [{M}, {G}], got {tuple(a_scale.shape)}")
    if b_scale.shape != (-(-N // 128), G):
        raise ValueError(f"b_scale must be [ceil(N / 128), ceil(K / 128)] = [{-(-N // 128)}, {G}], got {tuple(b_scale.shape)}")
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, 1)
        if bias.shape[0] != N:
            raise ValueError(f"bias must be [N] = [{N}]")
    if out_dtype not in _ROW_DTYPES:
        raise ValueError("out_dtype must be torch.bfloat16, torch.float16 or torch.float32")
    given = out
    if out is None:
        out = a.new_empty((M, N), dtype=out_dtype)
    else:
        _need(out, "out", out_dtype, 2)
        if out.shape != (M, N):
            raise ValueError(f"out must be [M, N] = [{M}, {N}]")
    _plain_operands("mm_fp8", "a", a, b=b, a_scale=a_scale, b_scale=b_scale, bias=bias, out=out)
    sm, sk = a_scale.stride()
    _call(_lib.nvfp4lora_mm_fp8, a.device, a.data_ptr(), b.data_ptr(), a_scale.data_ptr(), sm, sk, b_scale.data_ptr(),
          _ptr(bias), out.data_ptr(), _ROW_DTYPES[out_dtype], M, N, K)
    if given is not None:
        increment_version(given)
    return out
