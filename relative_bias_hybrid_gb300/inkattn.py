"""Thin ctypes binding of libinkattn.so (declared in include/inkattn.h).

Argument marshalling only: the entry points keep their C names, the params structs
mirror the C structs field by field, and the ``*_params`` helpers fill them from
torch tensors (device pointers, sizes).  Every step of the computation runs in the
library's CUDA kernels; there is no other implementation behind these calls, and
loading fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libinkattn.so")

INKATTN_OK = 0
INKATTN_ERR_INVALID_ARG = 1
INKATTN_ERR_UNSUPPORTED = 2
INKATTN_ERR_CUDA = 3
INKATTN_ERR_DEVICE_TIMEOUT = 4
INKATTN_ERR_DEVICE_BOUNDS = 5
INKATTN_DTYPE_BF16 = 0
INKATTN_DTYPE_F32 = 1
INKATTN_KV_BF16 = 0
INKATTN_KV_E4M3 = 1
INKATTN_KV_I4 = 4
INKATTN_ACT_NONE = 0
INKATTN_ACT_RELU = 1
INKATTN_ACT_GELU = 2
INKATTN_ACT_SILU = 3
INKATTN_ACT_SWIGLU = 4
INKATTN_SCORE_SIGMOID = 0
INKATTN_SCORE_SOFTMAX = 1

_c_i32 = ctypes.c_int32
_c_i64 = ctypes.c_int64
_c_ptr = ctypes.c_void_p


class PrologueParams(ctypes.Structure):
    """inkattn_prologue_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("B", _c_i32), ("N_tok", _c_i32), ("max_seqlen_q", _c_i32), ("Hq", _c_i32), ("Hkv", _c_i32),
        ("head_dim", _c_i32), ("block_size", _c_i32), ("num_blocks", _c_i32),
        ("num_state_slots", _c_i32), ("eps", ctypes.c_float),
        ("q", _c_ptr), ("k", _c_ptr), ("v", _c_ptr),
        ("conv_w_k", _c_ptr), ("conv_w_v", _c_ptr), ("q_norm_w", _c_ptr), ("k_norm_w", _c_ptr),
        ("cu_seqlens_q", _c_ptr), ("state_slot", _c_ptr), ("slot_mapping", _c_ptr),
        ("conv_state_k", _c_ptr), ("conv_state_v", _c_ptr), ("q_out", _c_ptr),
        ("k_cache", _c_ptr), ("v_cache", _c_ptr), ("kv_dtype", _c_i32), ("k_scale", _c_ptr),
        ("v_scale", _c_ptr), ("dev_status", _c_ptr),
    ]


class AttnParams(ctypes.Structure):
    """inkattn_attn_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("B", _c_i32), ("N_tok", _c_i32), ("max_seqlen_q", _c_i32), ("max_seqlen_k", _c_i32),
        ("Hq", _c_i32), ("Hkv", _c_i32), ("head_dim", _c_i32), ("block_size", _c_i32),
        ("num_blocks", _c_i32), ("max_blocks_per_seq", _c_i32), ("d_r", _c_i32),
        ("rel_extent", _c_i32), ("window", _c_i32), ("out_dtype", _c_i32),
        ("softmax_scale", ctypes.c_float), ("log_scale_base", ctypes.c_float),
        ("q", _c_ptr), ("r", _c_ptr), ("P", _c_ptr), ("k_cache", _c_ptr), ("v_cache", _c_ptr),
        ("kv_dtype", _c_i32), ("k_scale", _c_ptr), ("v_scale", _c_ptr), ("cu_seqlens_q", _c_ptr), ("seqlen_k", _c_ptr), ("block_table", _c_ptr),
        ("out", _c_ptr), ("lse", _c_ptr), ("dev_status", _c_ptr),
    ]


class OutputConvParams(ctypes.Structure):
    """inkattn_output_conv_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("B", _c_i32), ("N_tok", _c_i32), ("max_seqlen_q", _c_i32), ("D", _c_i32),
        ("num_state_slots", _c_i32), ("eps", ctypes.c_float),
        ("y", _c_ptr), ("conv_w", _c_ptr), ("norm_w", _c_ptr), ("cu_seqlens_q", _c_ptr),
        ("state_slot", _c_ptr), ("conv_state", _c_ptr), ("residual", _c_ptr), ("h_out", _c_ptr),
        ("out", _c_ptr), ("dev_status", _c_ptr),
    ]


class QkvrParams(ctypes.Structure):
    """inkattn_qkvr_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("B", _c_i32), ("N_tok", _c_i32), ("max_seqlen_q", _c_i32), ("Hq", _c_i32), ("Hkv", _c_i32),
        ("head_dim", _c_i32), ("d_r", _c_i32), ("d_model", _c_i32), ("block_size", _c_i32),
        ("num_blocks", _c_i32), ("num_state_slots", _c_i32), ("eps", ctypes.c_float),
        ("x", _c_ptr), ("w", _c_ptr),
        ("conv_w_k", _c_ptr), ("conv_w_v", _c_ptr), ("q_norm_w", _c_ptr), ("k_norm_w", _c_ptr),
        ("cu_seqlens_q", _c_ptr), ("state_slot", _c_ptr), ("slot_mapping", _c_ptr),
        ("conv_state_k_in", _c_ptr), ("conv_state_v_in", _c_ptr),
        ("conv_state_k_out", _c_ptr), ("conv_state_v_out", _c_ptr),
        ("q_out", _c_ptr), ("r_out", _c_ptr), ("y_out", _c_ptr),
        ("k_cache", _c_ptr), ("v_cache", _c_ptr), ("kv_dtype", _c_i32), ("k_scale", _c_ptr),
        ("v_scale", _c_ptr), ("dev_status", _c_ptr),
    ]


class LinearParams(ctypes.Structure):
    """inkattn_linear_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("N_tok", _c_i32), ("K", _c_i32), ("F", _c_i32), ("act", _c_i32), ("out_dtype", _c_i32),
        ("x", _c_ptr), ("w", _c_ptr), ("bias", _c_ptr), ("residual", _c_ptr), ("out", _c_ptr),
        ("dev_status", _c_ptr),
    ]


class GroupedLinearParams(ctypes.Structure):
    """inkattn_grouped_linear_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("E", _c_i32), ("M", _c_i32), ("N_x", _c_i32), ("K", _c_i32), ("F", _c_i32), ("act", _c_i32),
        ("out_dtype", _c_i32),
        ("x", _c_ptr), ("w", _c_ptr), ("bias", _c_ptr), ("expert_offsets", _c_ptr),
        ("row_token", _c_ptr), ("out", _c_ptr), ("dev_status", _c_ptr),
    ]


class RouteParams(ctypes.Structure):
    """inkattn_route_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("N_tok", _c_i32), ("E", _c_i32), ("n_shared", _c_i32), ("top_k", _c_i32), ("score", _c_i32),
        ("scale", ctypes.c_float),
        ("logits", _c_ptr), ("topk_ids", _c_ptr), ("weights", _c_ptr), ("expert_offsets", _c_ptr),
        ("row_token", _c_ptr), ("token_rows", _c_ptr),
    ]


class ExpertCombineParams(ctypes.Structure):
    """inkattn_expert_combine_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("N_tok", _c_i32), ("M", _c_i32), ("F", _c_i32), ("top_k", _c_i32), ("n_shared", _c_i32),
        ("y", _c_ptr), ("shared", _c_ptr), ("weights", _c_ptr), ("token_rows", _c_ptr), ("out", _c_ptr),
        ("dev_status", _c_ptr),
    ]


class TokenProbsParams(ctypes.Structure):
    """inkattn_token_probs_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("N_tok", _c_i32), ("V", _c_i32), ("logits_dtype", _c_i32),
        ("logits_stride", _c_i64), ("probs_stride", _c_i64),
        ("logits", _c_ptr), ("temperature", _c_ptr), ("probs", _c_ptr), ("dev_status", _c_ptr),
    ]


class VerifyDraftsParams(ctypes.Structure):
    """inkattn_verify_drafts_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("B", _c_i32), ("N_tok", _c_i32), ("V", _c_i32), ("target_stride", _c_i64), ("draft_stride", _c_i64),
        ("target_p", _c_ptr), ("draft_p", _c_ptr), ("token_ids", _c_ptr), ("cu_seqlens_q", _c_ptr),
        ("u_accept", _c_ptr), ("u_sample", _c_ptr), ("n_new", _c_ptr), ("out_tokens", _c_ptr),
        ("dev_status", _c_ptr),
    ]


class ConvRows(ctypes.Structure):
    """inkattn_conv_rows."""
    _fields_ = [("C", _c_i32), ("x_stride", _c_i64), ("x", _c_ptr), ("state_before", _c_ptr), ("state_after", _c_ptr)]


ROLLBACK_MAX_STATES = 8


class ConvRollbackParams(ctypes.Structure):
    """inkattn_conv_rollback_params."""
    _fields_ = [
        ("struct_size", ctypes.c_size_t),
        ("B", _c_i32), ("N_tok", _c_i32), ("num_state_slots", _c_i32), ("n_states", _c_i32),
        ("cu_seqlens_q", _c_ptr), ("state_slot", _c_ptr), ("n_keep", _c_ptr), ("dev_status", _c_ptr),
        ("states", ConvRows * ROLLBACK_MAX_STATES),
    ]


class InkattnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


_lock = threading.Lock()
_lib = None


def lib():
    """The loaded libinkattn.so.  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc)")
            L = ctypes.CDLL(LIB_PATH)
            P = ctypes.POINTER
            L.inkattn_status_string.argtypes = [ctypes.c_int]
            L.inkattn_status_string.restype = ctypes.c_char_p
            L.inkattn_abi_version.argtypes = []
            L.inkattn_abi_version.restype = ctypes.c_int
            L.inkattn_prologue.argtypes = [P(PrologueParams), _c_ptr]
            L.inkattn_prologue.restype = ctypes.c_int
            L.inkattn_prefill.argtypes = [P(AttnParams), _c_ptr]
            L.inkattn_prefill.restype = ctypes.c_int
            L.inkattn_decode_num_splits.argtypes = [P(AttnParams), ctypes.c_int]
            L.inkattn_decode_num_splits.restype = ctypes.c_int
            L.inkattn_decode_workspace_bytes.argtypes = [P(AttnParams), ctypes.c_int]
            L.inkattn_decode_workspace_bytes.restype = ctypes.c_size_t
            L.inkattn_decode.argtypes = [P(AttnParams), ctypes.c_int, _c_ptr, ctypes.c_size_t, _c_ptr]
            L.inkattn_decode.restype = ctypes.c_int
            L.inkattn_combine.argtypes = [P(AttnParams), ctypes.c_int, _c_ptr, ctypes.c_size_t, _c_ptr]
            L.inkattn_combine.restype = ctypes.c_int
            L.inkattn_decode_noalloc.argtypes = [P(AttnParams), ctypes.c_int, _c_ptr]
            L.inkattn_decode_noalloc.restype = ctypes.c_int
            L.inkattn_output_conv.argtypes = [P(OutputConvParams), _c_ptr]
            L.inkattn_output_conv.restype = ctypes.c_int
            L.inkattn_qkvr_prologue.argtypes = [P(QkvrParams), _c_ptr]
            L.inkattn_qkvr_prologue.restype = ctypes.c_int
            L.inkattn_prefill_workspace_bytes.argtypes = [P(AttnParams)]
            L.inkattn_prefill_workspace_bytes.restype = ctypes.c_size_t
            L.inkattn_prefill_e4m3.argtypes = [P(AttnParams), _c_ptr, ctypes.c_size_t, _c_ptr]
            L.inkattn_prefill_e4m3.restype = ctypes.c_int
            L.inkattn_prefill_i4.argtypes = [P(AttnParams), _c_ptr, ctypes.c_size_t, _c_ptr]
            L.inkattn_prefill_i4.restype = ctypes.c_int
            L.inkattn_linear.argtypes = [P(LinearParams), _c_ptr]
            L.inkattn_linear.restype = ctypes.c_int
            L.inkattn_grouped_linear.argtypes = [P(GroupedLinearParams), _c_ptr]
            L.inkattn_grouped_linear.restype = ctypes.c_int
            L.inkattn_route_workspace_bytes.argtypes = [P(RouteParams)]
            L.inkattn_route_workspace_bytes.restype = ctypes.c_size_t
            L.inkattn_route.argtypes = [P(RouteParams), _c_ptr, ctypes.c_size_t, _c_ptr]
            L.inkattn_route.restype = ctypes.c_int
            L.inkattn_expert_combine.argtypes = [P(ExpertCombineParams), _c_ptr]
            L.inkattn_expert_combine.restype = ctypes.c_int
            L.inkattn_token_probs.argtypes = [P(TokenProbsParams), _c_ptr]
            L.inkattn_token_probs.restype = ctypes.c_int
            L.inkattn_verify_drafts.argtypes = [P(VerifyDraftsParams), _c_ptr]
            L.inkattn_verify_drafts.restype = ctypes.c_int
            L.inkattn_conv_rollback.argtypes = [P(ConvRollbackParams), _c_ptr]
            L.inkattn_conv_rollback.restype = ctypes.c_int
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().inkattn_status_string(int(status)).decode()


def abi_version() -> int:
    return int(lib().inkattn_abi_version())


# The current stream's handle without building a torch.cuda.Stream for it (2.8 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(status: int, where: str, raise_on_error: bool):
    if raise_on_error and status != INKATTN_OK:
        raise InkattnError(status, where)
    return status


# ------------------------------------------------------------------ entry points

def inkattn_prologue(p: PrologueParams, stream=None, raise_on_error=True) -> int:
    return _check(lib().inkattn_prologue(ctypes.byref(p), _stream(stream)), "inkattn_prologue",
                  raise_on_error)


def inkattn_prefill(p: AttnParams, stream=None, raise_on_error=True) -> int:
    return _check(lib().inkattn_prefill(ctypes.byref(p), _stream(stream)), "inkattn_prefill",
                  raise_on_error)


def inkattn_prefill_workspace_bytes(p: AttnParams) -> int:
    return int(lib().inkattn_prefill_workspace_bytes(ctypes.byref(p)))


def inkattn_prefill_e4m3(p: AttnParams, workspace: Optional[torch.Tensor], stream=None,
                         raise_on_error=True) -> int:
    ptr, nbytes = _workspace(workspace)
    return _check(lib().inkattn_prefill_e4m3(ctypes.byref(p), ptr, nbytes, _stream(stream)),
                  "inkattn_prefill_e4m3", raise_on_error)


def inkattn_prefill_i4(p: AttnParams, workspace: Optional[torch.Tensor], stream=None, raise_on_error=True) -> int:
    ptr, nbytes = _workspace(workspace)
    return _check(lib().inkattn_prefill_i4(ctypes.byref(p), ptr, nbytes, _stream(stream)), "inkattn_prefill_i4",
                  raise_on_error)


def inkattn_decode_num_splits(p: AttnParams, num_sms: int) -> int:
    return int(lib().inkattn_decode_num_splits(ctypes.byref(p), int(num_sms)))


def inkattn_decode_workspace_bytes(p: AttnParams, num_splits: int) -> int:
    return int(lib().inkattn_decode_workspace_bytes(ctypes.byref(p), int(num_splits)))


def inkattn_decode(p: AttnParams, num_splits: int, workspace: Optional[torch.Tensor], stream=None,
                   raise_on_error=True) -> int:
    ptr, nbytes = _workspace(workspace)
    return _check(lib().inkattn_decode(ctypes.byref(p), int(num_splits), ptr, nbytes, _stream(stream)),
                  "inkattn_decode", raise_on_error)


def inkattn_combine(p: AttnParams, num_splits: int, workspace: Optional[torch.Tensor], stream=None,
                    raise_on_error=True) -> int:
    ptr, nbytes = _workspace(workspace)
    return _check(lib().inkattn_combine(ctypes.byref(p), int(num_splits), ptr, nbytes, _stream(stream)),
                  "inkattn_combine", raise_on_error)


DECODE_NOALLOC_MAX_BYTES = 64 << 20


def inkattn_decode_noalloc(p: AttnParams, num_splits: int, stream=None, raise_on_error=True) -> int:
    """Decode + combine with the split partials in the library's static device buffer
    (no workspace argument, no allocation): for callers that cannot allocate device
    memory where they decode."""
    return _check(lib().inkattn_decode_noalloc(ctypes.byref(p), int(num_splits), _stream(stream)),
                  "inkattn_decode_noalloc", raise_on_error)


def inkattn_output_conv(p: OutputConvParams, stream=None, raise_on_error=True) -> int:
    return _check(lib().inkattn_output_conv(ctypes.byref(p), _stream(stream)), "inkattn_output_conv",
                  raise_on_error)


# ------------------------------------------------------------------ marshalling helpers

def inkattn_qkvr_prologue(p: QkvrParams, stream=None, raise_on_error=True) -> int:
    return _check(lib().inkattn_qkvr_prologue(ctypes.byref(p), _stream(stream)), "inkattn_qkvr_prologue",
                  raise_on_error)


def inkattn_linear(p: LinearParams, stream=None, raise_on_error=True) -> int:
    return _check(lib().inkattn_linear(ctypes.byref(p), _stream(stream)), "inkattn_linear", raise_on_error)


def inkattn_grouped_linear(p: GroupedLinearParams, stream=None, raise_on_error=True) -> int:
    return _check(lib().inkattn_grouped_linear(ctypes.byref(p), _stream(stream)), "inkattn_grouped_linear",
                  raise_on_error)


def inkattn_route_workspace_bytes(p: RouteParams) -> int:
    return int(lib().inkattn_route_workspace_bytes(ctypes.byref(p)))


def inkattn_route(p: RouteParams, workspace: Optional[torch.Tensor] = None, stream=None,
                  raise_on_error=True) -> int:
    ptr, nbytes = _workspace(workspace)
    return _check(lib().inkattn_route(ctypes.byref(p), ptr, nbytes, _stream(stream)), "inkattn_route",
                  raise_on_error)


def inkattn_expert_combine(p: ExpertCombineParams, stream=None, raise_on_error=True) -> int:
    return _check(lib().inkattn_expert_combine(ctypes.byref(p), _stream(stream)), "inkattn_expert_combine",
                  raise_on_error)


def inkattn_token_probs(p: TokenProbsParams, stream=None, raise_on_error=True) -> int:
    return _check(lib().inkattn_token_probs(ctypes.byref(p), _stream(stream)), "inkattn_token_probs", raise_on_error)


def inkattn_verify_drafts(p: VerifyDraftsParams, stream=None, raise_on_error=True) -> int:
    return _check(lib().inkattn_verify_drafts(ctypes.byref(p), _stream(stream)), "inkattn_verify_drafts",
                  raise_on_error)


def inkattn_conv_rollback(p: ConvRollbackParams, stream=None, raise_on_error=True) -> int:
    return _check(lib().inkattn_conv_rollback(ctypes.byref(p), _stream(stream)), "inkattn_conv_rollback",
                  raise_on_error)


def _ptr(t: Optional[torch.Tensor], dtype=None, name="tensor") -> Optional[int]:
    if t is None:
        return None
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _workspace(t: Optional[torch.Tensor]):
    """Address and bytes of a workspace tensor.  One whose elements share memory (an expanded tensor)
    has fewer bytes than elements and is refused."""
    if t is None:
        return None, 0
    if not t.is_contiguous() and 1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())) < t.numel():
        raise ValueError("workspace: elements that share memory")
    return t.data_ptr(), t.numel() * t.element_size()


def _kv_dtype(cache, head_dim):
    """kv_dtype of a cache tensor: bf16 values, or codes held as uint8, a byte a value (E4M3) or
    half of one (4 bits)."""
    if cache.dtype == torch.bfloat16:
        return INKATTN_KV_BF16, torch.bfloat16
    if cache.dtype == torch.uint8:
        return (INKATTN_KV_I4 if 2 * cache.shape[-1] == head_dim else INKATTN_KV_E4M3), torch.uint8
    raise TypeError(f"KV cache: expected bfloat16 or uint8 (E4M3 or 4-bit codes), got {cache.dtype}")


def _kv_cache(p, k_cache, v_cache, k_scale, v_scale):
    """Fill the cache fields of a params struct: the codes' scales are fp32 [num_blocks][Hkv][64]
    (E4M3) or uint8 [num_blocks][Hkv][64][4] (4 bits)."""
    p.kv_dtype, dt = _kv_dtype(k_cache, p.head_dim)
    p.k_cache = _ptr(k_cache, dt, "k_cache"); p.v_cache = _ptr(v_cache, dt, "v_cache")
    if p.kv_dtype == INKATTN_KV_I4:
        rows = (p.num_blocks, p.Hkv, p.block_size)
        _one_device(k_cache, v_cache, k_scale, v_scale)
        for t, per, name in ((k_cache, 2, "k_cache"), (v_cache, 2, "v_cache"), (k_scale, 32, "k_scale"),
                             (v_scale, 32, "v_scale")):
            _shape(t, (*rows, p.head_dim // per), name)
        p.k_scale = _ptr(k_scale, torch.uint8, "k_scale"); p.v_scale = _ptr(v_scale, torch.uint8, "v_scale")
    elif p.kv_dtype == INKATTN_KV_E4M3:
        p.k_scale = _ptr(k_scale, torch.float32, "k_scale"); p.v_scale = _ptr(v_scale, torch.float32, "v_scale")


def prologue_params(*, q, k, v, conv_w_k, conv_w_v, q_norm_w, k_norm_w, cu_seqlens_q, state_slot,
                    slot_mapping, conv_state_k, conv_state_v, q_out, k_cache, v_cache,
                    max_seqlen_q: int, eps: float = 1e-6, dev_status=None, k_scale=None,
                    v_scale=None) -> PrologueParams:
    """Fill an inkattn_prologue_params from torch tensors (see include/inkattn.h)."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    N, Hq, d = q.shape
    Hkv = k.shape[1] // d
    p = PrologueParams()
    p.struct_size = ctypes.sizeof(PrologueParams)
    p.B = cu_seqlens_q.numel() - 1
    p.N_tok = N
    p.max_seqlen_q = int(max_seqlen_q)
    p.Hq, p.Hkv, p.head_dim = Hq, Hkv, d
    p.block_size = k_cache.shape[2]
    p.num_blocks = k_cache.shape[0]
    p.num_state_slots = conv_state_k.shape[0]
    p.eps = float(eps)
    p.q = _ptr(q, bf, "q"); p.k = _ptr(k, bf, "k"); p.v = _ptr(v, bf, "v")
    p.conv_w_k = _ptr(conv_w_k, f32, "conv_w_k"); p.conv_w_v = _ptr(conv_w_v, f32, "conv_w_v")
    p.q_norm_w = _ptr(q_norm_w, f32, "q_norm_w"); p.k_norm_w = _ptr(k_norm_w, f32, "k_norm_w")
    p.cu_seqlens_q = _ptr(cu_seqlens_q, i32, "cu_seqlens_q")
    p.state_slot = _ptr(state_slot, i32, "state_slot")
    p.slot_mapping = _ptr(slot_mapping, i32, "slot_mapping")
    p.conv_state_k = _ptr(conv_state_k, bf, "conv_state_k")
    p.conv_state_v = _ptr(conv_state_v, bf, "conv_state_v")
    p.q_out = _ptr(q_out, bf, "q_out")
    _kv_cache(p, k_cache, v_cache, k_scale, v_scale)
    p.dev_status = _ptr(dev_status, i32, "dev_status")
    return p


def attn_params(*, q, k_cache, v_cache, cu_seqlens_q, seqlen_k, block_table, out, max_seqlen_q: int,
                max_seqlen_k: int, r=None, P=None, rel_extent: int = 0, window: int = 0,
                softmax_scale: float = 0.0, log_scale_base: float = 0.0, lse=None,
                dev_status=None, k_scale=None, v_scale=None) -> AttnParams:
    """Fill an inkattn_attn_params from torch tensors (see include/inkattn.h)."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    N, Hq, d = q.shape
    p = AttnParams()
    p.struct_size = ctypes.sizeof(AttnParams)
    p.B = cu_seqlens_q.numel() - 1
    p.N_tok = N
    p.max_seqlen_q = int(max_seqlen_q)
    p.max_seqlen_k = int(max_seqlen_k)
    p.Hq, p.Hkv, p.head_dim = Hq, k_cache.shape[1], d
    p.block_size = k_cache.shape[2]
    p.num_blocks = k_cache.shape[0]
    p.max_blocks_per_seq = block_table.shape[1]
    p.d_r = r.shape[2] if r is not None else 0
    p.rel_extent = int(rel_extent)
    p.window = int(window)
    p.softmax_scale = float(softmax_scale)
    p.log_scale_base = float(log_scale_base)
    p.q = _ptr(q, bf, "q")
    p.r = _ptr(r, bf, "r") if rel_extent > 0 else None
    p.P = _ptr(P, f32, "P") if rel_extent > 0 else None
    _kv_cache(p, k_cache, v_cache, k_scale, v_scale)
    p.cu_seqlens_q = _ptr(cu_seqlens_q, i32, "cu_seqlens_q")
    p.seqlen_k = _ptr(seqlen_k, i32, "seqlen_k")
    p.block_table = _ptr(block_table, i32, "block_table")
    if out.dtype == torch.float32:
        p.out_dtype = INKATTN_DTYPE_F32
    elif out.dtype == bf:
        p.out_dtype = INKATTN_DTYPE_BF16
    else:
        raise TypeError(f"out: expected bfloat16 or float32, got {out.dtype}")
    p.out = _ptr(out, None, "out")
    p.lse = _ptr(lse, f32, "lse")
    p.dev_status = _ptr(dev_status, i32, "dev_status")
    return p


def output_conv_params(*, y, conv_w, norm_w, cu_seqlens_q, state_slot, conv_state, residual, h_out,
                       out, max_seqlen_q: int, eps: float = 1e-6, dev_status=None) -> OutputConvParams:
    """Fill an inkattn_output_conv_params from torch tensors (see include/inkattn.h)."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    N, D = y.shape
    p = OutputConvParams()
    p.struct_size = ctypes.sizeof(OutputConvParams)
    p.B = cu_seqlens_q.numel() - 1
    p.N_tok = N
    p.max_seqlen_q = int(max_seqlen_q)
    p.D = D
    p.num_state_slots = conv_state.shape[0]
    p.eps = float(eps)
    p.y = _ptr(y, bf, "y")
    p.conv_w = _ptr(conv_w, f32, "conv_w")
    p.norm_w = _ptr(norm_w, f32, "norm_w")
    p.cu_seqlens_q = _ptr(cu_seqlens_q, i32, "cu_seqlens_q")
    p.state_slot = _ptr(state_slot, i32, "state_slot")
    p.conv_state = _ptr(conv_state, bf, "conv_state")
    p.residual = _ptr(residual, bf, "residual")
    p.h_out = _ptr(h_out, bf, "h_out")
    p.out = _ptr(out, bf, "out")
    p.dev_status = _ptr(dev_status, i32, "dev_status")
    return p


def qkvr_params(*, x, w, conv_w_k, conv_w_v, q_norm_w, k_norm_w, cu_seqlens_q, state_slot, slot_mapping,
                conv_state_k_in, conv_state_v_in, conv_state_k_out, conv_state_v_out, q_out, r_out,
                k_cache, v_cache, max_seqlen_q: int, eps: float = 1e-6, dev_status=None, k_scale=None,
                v_scale=None, y_out=None) -> QkvrParams:
    """Fill an inkattn_qkvr_params from torch tensors (see include/inkattn.h): x [N][d_model],
    w [F][d_model], q_out [N][Hq][128], r_out [N][Hq][d_r], y_out None or [N][F]."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    N, Hq, d = q_out.shape
    p = QkvrParams()
    p.struct_size = ctypes.sizeof(QkvrParams)
    p.B = cu_seqlens_q.numel() - 1
    p.N_tok = N
    p.max_seqlen_q = int(max_seqlen_q)
    p.Hq, p.Hkv, p.head_dim = Hq, k_cache.shape[1], d
    p.d_r = r_out.shape[2]
    p.d_model = x.shape[1]
    p.block_size = k_cache.shape[2]
    p.num_blocks = k_cache.shape[0]
    p.num_state_slots = conv_state_k_in.shape[0]
    p.eps = float(eps)
    p.x = _ptr(x, bf, "x"); p.w = _ptr(w, bf, "w")
    p.conv_w_k = _ptr(conv_w_k, f32, "conv_w_k"); p.conv_w_v = _ptr(conv_w_v, f32, "conv_w_v")
    p.q_norm_w = _ptr(q_norm_w, f32, "q_norm_w"); p.k_norm_w = _ptr(k_norm_w, f32, "k_norm_w")
    p.cu_seqlens_q = _ptr(cu_seqlens_q, i32, "cu_seqlens_q")
    p.state_slot = _ptr(state_slot, i32, "state_slot")
    p.slot_mapping = _ptr(slot_mapping, i32, "slot_mapping")
    p.conv_state_k_in = _ptr(conv_state_k_in, bf, "conv_state_k_in")
    p.conv_state_v_in = _ptr(conv_state_v_in, bf, "conv_state_v_in")
    p.conv_state_k_out = _ptr(conv_state_k_out, bf, "conv_state_k_out")
    p.conv_state_v_out = _ptr(conv_state_v_out, bf, "conv_state_v_out")
    p.q_out = _ptr(q_out, bf, "q_out"); p.r_out = _ptr(r_out, bf, "r_out")
    p.y_out = _ptr(y_out, bf, "y_out")
    _kv_cache(p, k_cache, v_cache, k_scale, v_scale)
    p.dev_status = _ptr(dev_status, i32, "dev_status")
    return p


ACTIVATIONS = {"none": INKATTN_ACT_NONE, "relu": INKATTN_ACT_RELU, "gelu": INKATTN_ACT_GELU,
               "silu": INKATTN_ACT_SILU, "swiglu": INKATTN_ACT_SWIGLU}
SCORES = {"sigmoid": INKATTN_SCORE_SIGMOID, "softmax": INKATTN_SCORE_SOFTMAX}


def _out_dtype(out):
    if out.dtype == torch.float32:
        return INKATTN_DTYPE_F32
    if out.dtype == torch.bfloat16:
        return INKATTN_DTYPE_BF16
    raise TypeError(f"out: expected bfloat16 or float32, got {out.dtype}")


def _shape(t, shape, name):
    """The sizes a params struct holds once must be those of every tensor that has them."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _one_device(*tensors):
    """A call's tensors lie on one device; the library compares it with the current one."""
    devices = {t.device for t in tensors if t is not None}
    if len(devices) > 1:
        raise ValueError(f"tensors on several devices: {sorted(map(str, devices))}")


def linear_params(*, x, w, out, act: str = "none", bias=None, residual=None, dev_status=None) -> LinearParams:
    """Fill an inkattn_linear_params from torch tensors (see include/inkattn.h): x [N][K],
    w [F][K] (act "swiglu": [2F][K], the gate rows first), bias fp32 None or one per row of w,
    residual None or [N][F], out [N][F] bf16 or fp32."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    N, K = x.shape
    F = out.shape[1]
    rows = 2 * F if act == "swiglu" else F
    _one_device(x, w, out, bias, residual, dev_status)
    _shape(w, (rows, K), "w"); _shape(out, (N, F), "out"); _shape(bias, (rows,), "bias")
    _shape(residual, (N, F), "residual")
    p = LinearParams()
    p.struct_size = ctypes.sizeof(LinearParams)
    p.N_tok, p.K, p.F = N, K, F
    p.act = ACTIVATIONS[act]
    p.out_dtype = _out_dtype(out)
    p.x = _ptr(x, bf, "x"); p.w = _ptr(w, bf, "w")
    p.bias = _ptr(bias, f32, "bias"); p.residual = _ptr(residual, bf, "residual")
    p.out = _ptr(out, None, "out")
    p.dev_status = _ptr(dev_status, i32, "dev_status")
    p.tensors = (x, w, out, bias, residual, dev_status)     # alive as long as the params
    return p


def grouped_linear_params(*, x, w, expert_offsets, out, act: str = "none", row_token=None, bias=None,
                          dev_status=None) -> GroupedLinearParams:
    """Fill an inkattn_grouped_linear_params from torch tensors (see include/inkattn.h):
    x [N_x][K], w [E][F][K] (act "swiglu": [E][2F][K]), expert_offsets [E+1], row_token None or
    [M], bias None or [E][rows of w], out [M][F] bf16 or fp32."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    N_x, K = x.shape
    M, F = out.shape
    E = w.shape[0]
    rows = 2 * F if act == "swiglu" else F
    _one_device(x, w, expert_offsets, out, row_token, bias, dev_status)
    _shape(w, (E, rows, K), "w"); _shape(expert_offsets, (E + 1,), "expert_offsets")
    _shape(row_token, (M,), "row_token"); _shape(bias, (E, rows), "bias")
    p = GroupedLinearParams()
    p.struct_size = ctypes.sizeof(GroupedLinearParams)
    p.E, p.M, p.N_x, p.K, p.F = E, M, N_x, K, F
    p.act = ACTIVATIONS[act]
    p.out_dtype = _out_dtype(out)
    p.x = _ptr(x, bf, "x"); p.w = _ptr(w, bf, "w"); p.bias = _ptr(bias, f32, "bias")
    p.expert_offsets = _ptr(expert_offsets, i32, "expert_offsets")
    p.row_token = _ptr(row_token, i32, "row_token")
    p.out = _ptr(out, None, "out")
    p.dev_status = _ptr(dev_status, i32, "dev_status")
    p.tensors = (x, w, expert_offsets, out, row_token, bias, dev_status)     # alive as long as the params
    return p


def route_params(*, logits, topk_ids, weights, expert_offsets, row_token, token_rows, n_shared: int = 0,
                 score: str = "sigmoid", scale: float = 1.0) -> RouteParams:
    """Fill an inkattn_route_params from torch tensors (see include/inkattn.h): logits
    [N][E + n_shared], topk_ids [N][k], weights [N][k + n_shared], expert_offsets [E+1],
    row_token [N*k], token_rows [N][k]."""
    f32, i32 = torch.float32, torch.int32
    N, k = topk_ids.shape
    E = logits.shape[1] - int(n_shared)
    _one_device(logits, topk_ids, weights, expert_offsets, row_token, token_rows)
    _shape(logits, (N, E + n_shared), "logits"); _shape(weights, (N, k + n_shared), "weights")
    _shape(expert_offsets, (E + 1,), "expert_offsets"); _shape(row_token, (N * k,), "row_token")
    _shape(token_rows, (N, k), "token_rows")
    p = RouteParams()
    p.struct_size = ctypes.sizeof(RouteParams)
    p.N_tok, p.E, p.n_shared, p.top_k = N, E, int(n_shared), k
    p.score = SCORES[score]
    p.scale = float(scale)
    p.logits = _ptr(logits, f32, "logits"); p.topk_ids = _ptr(topk_ids, i32, "topk_ids")
    p.weights = _ptr(weights, f32, "weights")
    p.expert_offsets = _ptr(expert_offsets, i32, "expert_offsets")
    p.row_token = _ptr(row_token, i32, "row_token"); p.token_rows = _ptr(token_rows, i32, "token_rows")
    p.tensors = (logits, topk_ids, weights, expert_offsets, row_token, token_rows)     # alive as long as the params
    return p


def expert_combine_params(*, y, weights, token_rows, out, shared=None, dev_status=None) -> ExpertCombineParams:
    """Fill an inkattn_expert_combine_params from torch tensors (see include/inkattn.h): y [M][F],
    weights [N][k + n_shared], token_rows [N][k], shared None or [n_shared][N][F], out [N][F]."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    M, F = y.shape
    N, k = token_rows.shape
    S = shared.shape[0] if shared is not None else 0
    _one_device(y, weights, token_rows, out, shared, dev_status)
    _shape(weights, (N, k + S), "weights"); _shape(out, (N, F), "out"); _shape(shared, (S, N, F), "shared")
    p = ExpertCombineParams()
    p.struct_size = ctypes.sizeof(ExpertCombineParams)
    p.N_tok, p.M, p.F, p.top_k, p.n_shared = N, M, F, k, S
    p.y = _ptr(y, bf, "y"); p.shared = _ptr(shared, bf, "shared"); p.weights = _ptr(weights, f32, "weights")
    p.token_rows = _ptr(token_rows, i32, "token_rows"); p.out = _ptr(out, bf, "out")
    p.dev_status = _ptr(dev_status, i32, "dev_status")
    p.tensors = (y, weights, token_rows, out, shared, dev_status)     # alive as long as the params
    return p


def _rows(t: Optional[torch.Tensor], dtype, name):
    """Address and row stride of a matrix whose rows are dense, possibly a part of wider rows."""
    if t is None:
        return None, 0
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"{name}: expected rows of adjacent elements that do not overlap")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else t.shape[1]


def token_probs_params(*, logits, probs, temperature=None, dev_status=None) -> TokenProbsParams:
    """Fill an inkattn_token_probs_params from torch tensors (see include/inkattn.h): logits [N][V]
    bf16 or fp32, probs [N][V] fp32 (either may be columns of wider rows; probs may be logits),
    temperature None or [N] fp32."""
    N, V = logits.shape
    _one_device(logits, probs, temperature, dev_status)
    _shape(probs, (N, V), "probs"); _shape(temperature, (N,), "temperature")
    p = TokenProbsParams()
    p.struct_size = ctypes.sizeof(TokenProbsParams)
    p.N_tok, p.V = N, V
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits: expected bfloat16 or float32, got {logits.dtype}")
    p.logits_dtype = INKATTN_DTYPE_F32 if logits.dtype == torch.float32 else INKATTN_DTYPE_BF16
    p.logits, p.logits_stride = _rows(logits, None, "logits")
    p.probs, p.probs_stride = _rows(probs, torch.float32, "probs")
    p.temperature = _ptr(temperature, torch.float32, "temperature")
    p.dev_status = _ptr(dev_status, torch.int32, "dev_status")
    p.tensors = (logits, probs, temperature, dev_status)     # alive as long as the params
    return p


def verify_drafts_params(*, target_p, token_ids, cu_seqlens_q, u_accept, u_sample, n_new, out_tokens, draft_p=None,
                         dev_status=None) -> VerifyDraftsParams:
    """Fill an inkattn_verify_drafts_params from torch tensors (see include/inkattn.h): target_p [N][V]
    fp32, draft_p None or [N][V] fp32 (either may be columns of wider rows), token_ids [N],
    cu_seqlens_q [B+1], u_accept [N], u_sample [B], n_new [B], out_tokens [N]."""
    f32, i32 = torch.float32, torch.int32
    N, V = target_p.shape
    B = cu_seqlens_q.numel() - 1
    _one_device(target_p, draft_p, token_ids, cu_seqlens_q, u_accept, u_sample, n_new, out_tokens, dev_status)
    _shape(draft_p, (N, V), "draft_p"); _shape(token_ids, (N,), "token_ids"); _shape(u_accept, (N,), "u_accept")
    _shape(cu_seqlens_q, (B + 1,), "cu_seqlens_q"); _shape(u_sample, (B,), "u_sample"); _shape(n_new, (B,), "n_new")
    _shape(out_tokens, (N,), "out_tokens")
    p = VerifyDraftsParams()
    p.struct_size = ctypes.sizeof(VerifyDraftsParams)
    p.B, p.N_tok, p.V = B, N, V
    p.target_p, p.target_stride = _rows(target_p, f32, "target_p")
    p.draft_p, p.draft_stride = _rows(draft_p, f32, "draft_p")
    p.token_ids = _ptr(token_ids, i32, "token_ids"); p.cu_seqlens_q = _ptr(cu_seqlens_q, i32, "cu_seqlens_q")
    p.u_accept = _ptr(u_accept, f32, "u_accept"); p.u_sample = _ptr(u_sample, f32, "u_sample")
    p.n_new = _ptr(n_new, i32, "n_new"); p.out_tokens = _ptr(out_tokens, i32, "out_tokens")
    p.dev_status = _ptr(dev_status, i32, "dev_status")
    p.tensors = (target_p, draft_p, token_ids, cu_seqlens_q, u_accept, u_sample, n_new, out_tokens, dev_status)
    return p


def conv_rollback_params(*, x, state_before, state_after, n_keep, cu_seqlens_q, state_slot,
                         dev_status=None) -> ConvRollbackParams:
    """Fill an inkattn_conv_rollback_params from torch tensors (see include/inkattn.h): lists of one to
    eight convs' tensors, x [N][C] bf16 (possibly columns of wider rows), state_before and state_after
    [num_state_slots][3][C] bf16; n_keep [B], cu_seqlens_q [B+1], state_slot [B]."""
    bf, i32 = torch.bfloat16, torch.int32
    if not 1 <= len(x) <= ROLLBACK_MAX_STATES or len(state_before) != len(x) or len(state_after) != len(x):
        raise ValueError(f"conv states: expected one to {ROLLBACK_MAX_STATES}, as many of each")
    B, N, slots = cu_seqlens_q.numel() - 1, x[0].shape[0], state_before[0].shape[0]
    _one_device(*x, *state_before, *state_after, n_keep, cu_seqlens_q, state_slot, dev_status)
    _shape(cu_seqlens_q, (B + 1,), "cu_seqlens_q"); _shape(state_slot, (B,), "state_slot"); _shape(n_keep, (B,), "n_keep")
    p = ConvRollbackParams()
    p.struct_size = ctypes.sizeof(ConvRollbackParams)
    p.B, p.N_tok, p.num_state_slots, p.n_states = B, N, slots, len(x)
    p.cu_seqlens_q = _ptr(cu_seqlens_q, i32, "cu_seqlens_q"); p.state_slot = _ptr(state_slot, i32, "state_slot")
    p.n_keep = _ptr(n_keep, i32, "n_keep"); p.dev_status = _ptr(dev_status, i32, "dev_status")
    for c, xs, before, after in zip(p.states, x, state_before, state_after):
        c.C = before.shape[2]
        _shape(xs, (N, c.C), "x"); _shape(before, (slots, 3, c.C), "state_before"); _shape(after, (slots, 3, c.C), "state_after")
        c.x, c.x_stride = _rows(xs, bf, "x")
        c.state_before = _ptr(before, bf, "state_before"); c.state_after = _ptr(after, bf, "state_after")
    p.tensors = (*x, *state_before, *state_after, n_keep, cu_seqlens_q, state_slot, dev_status)     # alive as long as the params
    return p
