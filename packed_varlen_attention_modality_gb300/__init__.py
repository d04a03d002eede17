"""GB300-native packed varlen attention with modality-tagged 3D RoPE.

Thin Python binding over the C ABI of ``libh3attn.so`` (declared in include/h3attn.h).  It only
marshals arguments -- checks dtypes and shapes, takes device pointers and the current CUDA
stream from PyTorch tensors -- and every step of the computation runs in the library's CUDA
kernels.  There is no CPU or PyTorch fallback: if the library is missing, every call raises.

Calls:
  rope_apply        modality-tagged RoPE of Q and K with the continuation time shift
  qk_norm_rope / qk_norm_rope_bwd   RMS norm of Q and K per head with the rotation (or without)
                    in the same pass, and its gradient
  residual_norm / residual_norm_bwd   the step between two branches of a block: gated residual with an
                    optional norm of the branch, then the modulated norm of the stream; and its gradient
  varlen_attn_fwd   block-diagonal softmax attention over cu_seqlens segments
  varlen_cross_attn_fwd / varlen_cross_attn_bwd   packed cross attention: keys of another length per
                    segment, query heads sharing key heads, padded key batches; and its gradient
                    (with equal offsets, that of varlen_attn_fwd)
  kv_cache_write / kv_cache_read   rows of keys and values into a paged cache (bf16, or e4m3 with a
                    power-of-two scale per row), and back out of it
  paged_attn_fwd    attention of new tokens (single ones or chunks) over a paged cache, causal by token or
                    by blocks of tokens
  window_count / window_pack / window_unpack   shifted 3D window partition and row gather/scatter
  window_attn_fwd   shifted 3D window attention read and written in place on the grid
  vsa_select / vsa_attn_fwd   block-sparse video attention: block gate scores + top-k
                    selection, then attention over the selected 64-token blocks (paired query
                    blocks share the key blocks both selected)
  continuation_plan / continuation_pack / continuation_append / masked_row_update
                    continuation window: tails, five row groups, overlap discard, target updates
  sp_assign_windows / sp_rank_tokens / sp_layer_order / sp_exchange_plan
                    window-aligned sequence parallelism: window owners, local orders and the
                    all-to-all plan of a regular <-> shifted switch (host planning; the caller
                    moves the rows with its own all-to-all)
  get_device_error  read (and clear) the device-side error word
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

__all__ = ["H3Error", "RopeConfig", "lib_path", "load_library", "rope_apply", "qk_norm_rope",
           "qk_norm_rope_bwd_workspace_size", "qk_norm_rope_bwd", "residual_norm", "ResidualNormGrads",
           "residual_norm_bwd_workspace_size", "residual_norm_bwd", "kv_cache_write", "kv_cache_read",
           "paged_attn_workspace_size", "paged_attn_fwd",
           "varlen_attn_fwd",
           "varlen_attn_fwd_noalloc", "varlen_cross_attn_workspace_size", "varlen_cross_attn_fwd",
           "varlen_cross_attn_bwd_workspace_size", "varlen_cross_attn_bwd",
           "window_attn_fwd", "vsa_block_count",
           "vsa_select_workspace_size", "vsa_select", "vsa_attn_workspace_size", "vsa_attn_fwd",
           "ContinuationConfig",
           "ContinuationPlan", "continuation_config", "continuation_plan", "continuation_pack",
           "continuation_append", "masked_row_update", "sp_assign_windows", "sp_layer_order",
           "sp_rank_tokens", "sp_exchange_plan",
           "varlen_attn_workspace_size", "window_count", "window_pack", "window_unpack",
           "get_device_error", "TAG_TEXT", "TAG_VIDEO", "TAG_AUDIO"]

TAG_TEXT, TAG_VIDEO, TAG_AUDIO = 0, 1, 2

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libh3attn.so"
_lib = None

_STATUS = {0: "H3_OK", 1: "H3_ERR_NULL", 2: "H3_ERR_INVALID_ARG", 3: "H3_ERR_BAD_CU_SEQLENS",
           4: "H3_ERR_UNSUPPORTED", 5: "H3_ERR_WORKSPACE", 6: "H3_ERR_CUDA", 7: "H3_ERR_TIMEOUT",
           8: "H3_ERR_MISALIGNED", 9: "H3_ERR_BAD_PERM", 10: "H3_ERR_BAD_BLOCK_INDEX",
           11: "H3_ERR_SMEM_LAYOUT", 12: "H3_ERR_BAD_PAGE"}


class H3Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        self.name = _STATUS.get(self.status, f"status {status}")
        msg = load_library().h3_status_string(self.status).decode()
        super().__init__(f"{where}: {self.name}: {msg}")


class RopeConfig(ctypes.Structure):
    """Mirror of h3_rope_cfg; zero fields select the defaults (base 10000, D/2:D/4:D/4, 40/24)."""
    _fields_ = [("base_text", ctypes.c_float), ("base_video", ctypes.c_float),
                ("base_audio", ctypes.c_float), ("video_dims_t", ctypes.c_int32),
                ("video_dims_h", ctypes.c_int32), ("video_dims_w", ctypes.c_int32),
                ("audio_hz", ctypes.c_float), ("video_fps", ctypes.c_float)]


_I = ctypes.c_int32


_L = ctypes.c_int64


class _QkNormDesc(ctypes.Structure):
    """Mirror of h3_qk_norm_desc."""
    _fields_ = [("num_tokens", _I), ("num_q_heads", _I), ("num_k_heads", _I), ("head_dim", _I),
                ("weight_type", _I), ("eps", ctypes.c_float), ("q_stride", _L), ("k_stride", _L),
                ("q_out_stride", _L), ("k_out_stride", _L), ("dq_stride", _L), ("dk_stride", _L)]
    pack = struct.Struct("@5if6q").pack  # the same bytes, several times faster than the class


class _ResidualNormDesc(ctypes.Structure):
    """Mirror of h3_residual_norm_desc."""
    _fields_ = [("num_tokens", _I), ("dim", _I), ("num_requests", _I), ("norm", _I), ("branch_norm", _I),
                ("stream_type", _I), ("weight_type", _I), ("mod_type", _I), ("eps", ctypes.c_float),
                ("residual_scale", ctypes.c_float), ("x_stride", _L), ("y_stride", _L), ("x_out_stride", _L),
                ("h_stride", _L), ("scale_stride", _L), ("shift_stride", _L), ("gate_stride", _L),
                ("dx_out_stride", _L), ("dh_stride", _L), ("dx_stride", _L), ("dy_stride", _L)]
    pack = struct.Struct("@8i2f11q").pack


class _KvCacheDesc(ctypes.Structure):
    """Mirror of h3_kv_cache_desc."""
    _fields_ = [("num_segments", _I), ("capacity", _I), ("num_heads", _I), ("head_dim", _I), ("cache_type", _I),
                ("page_size", _I), ("num_pages", _I), ("max_pages", _I), ("k_stride", _L), ("v_stride", _L)]
    pack = struct.Struct("@8i2q").pack


class _PagedAttnDesc(ctypes.Structure):
    """Mirror of h3_paged_attn_desc."""
    _fields_ = [("num_segments", _I), ("max_seqlen_q", _I), ("max_seqlen_k", _I), ("capacity_q", _I),
                ("num_q_heads", _I), ("num_kv_heads", _I), ("head_dim", _I), ("cache_type", _I), ("page_size", _I),
                ("num_pages", _I), ("max_pages", _I), ("causal_block", _I), ("softmax_scale", ctypes.c_float),
                ("q_stride", _L)]
    pack = struct.Struct("@12ifq").pack


class _CrossAttnDesc(ctypes.Structure):
    """Mirror of h3_cross_attn_desc."""
    _fields_ = [("num_segments", _I), ("max_seqlen_q", _I), ("max_seqlen_k", _I), ("capacity_q", _I),
                ("capacity_k", _I), ("num_q_heads", _I), ("num_kv_heads", _I), ("head_dim", _I),
                ("softmax_scale", ctypes.c_float), ("q_stride", _L), ("k_stride", _L), ("v_stride", _L),
                ("dq_stride", _L), ("dk_stride", _L), ("dv_stride", _L)]
    pack = struct.Struct("@8if4x6q").pack


class ContinuationConfig(ctypes.Structure):
    """Mirror of h3_continuation_cfg."""
    _fields_ = [("text_rows", _I), ("clip_video_frames", _I), ("clip_audio_rows", _I),
                ("frame_h", _I), ("frame_w", _I), ("new_video_frames", _I), ("new_audio_rows", _I),
                ("tail_frames", _I), ("frames_per_latent", _I)]


class ContinuationPlan(ctypes.Structure):
    """Mirror of h3_continuation_plan."""
    _fields_ = [("tail_start", _I), ("start_frame", _I), ("audio_cut", _I), ("group_rows", _I * 5),
                ("group_offset", _I * 6), ("num_rows", _I), ("keep_video_from", _I),
                ("keep_audio_from", _I), ("out_video_frames", _I), ("out_audio_rows", _I)]


def lib_path() -> str:
    return os.path.join(_PKG_DIR, _LIB_NAME)


def load_library():
    """Load libh3attn.so (built in-tree by __graft_entry__.build()); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -c 'import __graft_entry__ as g; "
                           "g.build()'` first (this package has no CPU fallback)")
    lib = ctypes.CDLL(path)
    P, I32, U64, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    I32P = ctypes.POINTER(ctypes.c_int32)
    sigs = {
        "h3_rope_apply": (I32, [P, P, P, P, I32, I32, I32, P, P, P, I32, P,
                                ctypes.POINTER(RopeConfig), P]),
        "h3_qk_norm_rope": (I32, [P, P, P, P, P, P, P, P, P, P, I32, P,
                                  ctypes.POINTER(RopeConfig), P]),
        "h3_qk_norm_rope_bwd_workspace_size": (U64, [I32]),
        "h3_qk_norm_rope_bwd": (I32, [P, P, P, P, P, P, P, P, P, P, I32, P,
                                      ctypes.POINTER(RopeConfig), P, P, P, P, P, U64, P]),
        "h3_residual_norm": (I32, [P] * 12),
        "h3_residual_norm_bwd_workspace_size": (U64, [P]),
        "h3_residual_norm_bwd": (I32, [P] * 18 + [U64, P]),
        "h3_kv_cache_write": (I32, [P] * 11),
        "h3_kv_cache_read": (I32, [P] * 11),
        "h3_paged_attn_workspace_size": (U64, [P]),
        "h3_paged_attn_fwd": (I32, [P] * 12 + [U64, P]),
        "h3_varlen_attn_workspace_size": (U64, [I32, I32, I32, I32]),
        "h3_varlen_attn_fwd": (I32, [P, P, P, P, P, P, I32, I32, I32, I32, I32, F32, P, U64, P]),
        "h3_varlen_attn_fwd_noalloc": (I32, [P, P, P, P, P, P, I32, I32, I32, I32, I32, F32, P]),
        "h3_varlen_cross_attn_workspace_size": (U64, [P]),
        "h3_varlen_cross_attn_fwd": (I32, [P, P, P, P, P, P, P, P, P, P, U64, P]),
        "h3_varlen_cross_attn_bwd_workspace_size": (U64, [P]),
        "h3_varlen_cross_attn_bwd": (I32, [P, P, P, P, P, P, P, P, P, P, P, P, P, P,
                                           U64, P]),
        "h3_window_attn_fwd": (I32, [P, P, P, P, P, I32P, I32P, I32P, I32, I32, F32, P]),
        "h3_window_count": (I32, [I32P, I32P, I32P]),
        "h3_window_pack": (I32, [I32P, I32P, I32P, P, P, ctypes.POINTER(P), ctypes.POINTER(P),
                                 I32, I32, P]),
        "h3_window_unpack": (I32, [P, I32, P, P, I32, P]),
        "h3_vsa_block_count": (I32, [I32P, I32P]),
        "h3_continuation_make_plan": (I32, [ctypes.POINTER(ContinuationConfig), ctypes.POINTER(ContinuationPlan)]),
        "h3_continuation_pack": (I32, [ctypes.POINTER(ContinuationConfig), P, P, P, P, P, I32, P, P, P, P, P]),
        "h3_continuation_append": (I32, [ctypes.POINTER(ContinuationConfig), P, P, I32, P, ctypes.c_int64, P,
                                         ctypes.c_int64, P]),
        "h3_masked_row_update": (I32, [P, P, P, I32, I32, P]),
        "h3_sp_assign_windows": (I32, [I32P, I32P, I32P, I32, P, P]),
        "h3_sp_rank_tokens": (I32, [I32P, I32P, I32P, P, I32, P]),
        "h3_sp_layer_order": (I32, [I32P, I32P, I32P, P, I32, I32, P, ctypes.c_int64]),
        "h3_sp_exchange_plan": (I32, [I32P, I32P, I32P, P, I32P, P, I32, I32, P, P, P, P]),
        "h3_vsa_select_workspace_size": (U64, [I32P, I32P, I32, I32]),
        "h3_vsa_select": (I32, [P, P, I32P, I32P, I32, I32, I32, F32, P, P, P, U64, P]),
        "h3_vsa_attn_workspace_size": (U64, [I32P, I32P, I32, I32]),
        "h3_vsa_attn_fwd": (I32, [P, P, P, P, P, I32P, I32P, I32, I32, P, I32, F32, P, U64, P]),
        "h3_set_wait_limit_ns": (ctypes.c_uint64, [ctypes.c_uint64]),
        "h3_debug_stall_loads": (I32, [I32]),
        "h3_get_device_error": (I32, [P]),
        "h3_status_string": (ctypes.c_char_p, [I32]),
        "h3_version": (I32, []),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != 0:
        raise H3Error(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _launch(fn, where: str, device: torch.device, *args):
    """Call a launching entry point on `device`'s current stream; raise on a failed status."""
    index = device.index
    if index == torch.cuda.current_device():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != 0:
        raise H3Error(st, where)


def _require(t: torch.Tensor, name: str, dtype, device: torch.device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _i3(v: Sequence[int]):
    a = (ctypes.c_int32 * 3)(*[int(x) for x in v])
    return a


def rope_apply(q: torch.Tensor, k: Optional[torch.Tensor], pos: torch.Tensor, tag: torch.Tensor,
               cu_requests: Optional[torch.Tensor] = None, start_frames: Optional[torch.Tensor] = None,
               num_tokens: Optional[int] = None, q_out: Optional[torch.Tensor] = None,
               k_out: Optional[torch.Tensor] = None, cfg: Optional[RopeConfig] = None):
    """Tagged RoPE of q (and k) [C, H, D] bf16; in place unless q_out / k_out are given.

    pos fp32 [>=N, 3] (t, h, w); tag uint8 [>=N]; cu_requests int32 [R+1] and start_frames fp32
    [R] (continuation start frames s_r) are optional.  Returns (q_out, k_out).
    """
    dev = q.device
    _require(q, "q", torch.bfloat16, dev)
    if q.dim() != 3:
        raise ValueError("q must be [C, H, D]")
    C, H, D = q.shape
    n = C if num_tokens is None else int(num_tokens)
    if n > C:
        raise ValueError("num_tokens exceeds the capacity of q")
    q_out = q if q_out is None else q_out
    _require(q_out, "q_out", torch.bfloat16, dev)
    if k is not None:
        _require(k, "k", torch.bfloat16, dev)
        k_out = k if k_out is None else k_out
        _require(k_out, "k_out", torch.bfloat16, dev)
        if k.shape != q.shape or k_out.shape != q.shape:
            raise ValueError("k must have q's shape")
    else:
        k_out = None
    if q_out.shape != q.shape:
        raise ValueError("q_out must have q's shape")
    _require(pos, "pos", torch.float32, dev)
    _require(tag, "tag", torch.uint8, dev)
    if pos.shape[0] < n or tag.shape[0] < n:
        raise ValueError("pos / tag must cover num_tokens rows")
    nreq = 0
    if cu_requests is not None:
        _require(cu_requests, "cu_requests", torch.int32, dev)
        nreq = cu_requests.numel() - 1
    if start_frames is not None:
        _require(start_frames, "start_frames", torch.float32, dev)
        if cu_requests is not None and start_frames.numel() < nreq:
            raise ValueError("start_frames must have one entry per request")
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.h3_rope_apply(_ptr(q), _ptr(q_out), _ptr(k), _ptr(k_out), n, H, D, _ptr(pos),
                               _ptr(tag), _ptr(cu_requests), nreq, _ptr(start_frames),
                               ctypes.byref(cfg) if cfg is not None else None, _stream(dev))
    _check(st, "h3_rope_apply")
    return q_out, k_out


_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _aux(t: torch.Tensor, name: str, dtype, device: torch.device):
    """_require, its common case first."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.is_contiguous()):
        _require(t, name, dtype, device)


def _rows(t: torch.Tensor, name: str, device: torch.device, shape=None) -> int:
    """Check bf16 [C, H, D] rows with heads and dims contiguous (a part of a fused projection is
    fine); returns the token stride in elements, 0 for contiguous rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be {_BF16}, got {t.dtype}")
    C, H, D = shape3 = t.shape if t.dim() == 3 else (None, None, None)
    if C is None:
        raise ValueError(f"{name} must be [C, H, D]")
    if shape is not None and shape3 != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.is_contiguous():
        return 0
    sc, sh, sd = t.stride()
    if sd != 1 or (H > 1 and sh != D) or (C > 1 and sc < H * D):
        raise ValueError(f"{name} must have contiguous heads and dims within a token")
    return sc if C > 1 else 0


def _norm_inputs(q, k, q_weight, k_weight, pos, tag, cu_requests, start_frames, num_tokens):
    """Checks shared by qk_norm_rope and its backward; returns (num_requests, pointers of the rotation's
    inputs, sizes of the descriptor, q and k strides)."""
    dev = q.device
    q_stride, k_stride, hk = _rows(q, "q", dev), 0, 0
    C, H, D = q.shape
    n = C if num_tokens is None else int(num_tokens)
    if not 0 <= n <= C:
        raise ValueError("num_tokens must lie within the capacity of q")
    kind = q_weight.dtype if isinstance(q_weight, torch.Tensor) else None
    if kind is not _F32 and kind is not _BF16:
        raise TypeError("q_weight must be a float32 or bfloat16 tensor")
    _aux(q_weight, "q_weight", kind, dev)
    if q_weight.shape != (D,):
        raise ValueError("q_weight must be [head_dim]")
    if k is not None:
        k_stride = _rows(k, "k", dev)
        Ck, hk, Dk = k.shape
        if Ck != C or Dk != D:
            raise ValueError("k must have q's tokens and head_dim")
        _aux(k_weight, "k_weight", kind, dev)
        if k_weight.shape != (D,):
            raise ValueError("k_weight must be [head_dim]")
    nreq = 0
    if (pos is None) != (tag is None):
        raise ValueError("pos and tag are given together")
    if pos is None:
        if cu_requests is not None or start_frames is not None:
            raise ValueError("cu_requests and start_frames need pos and tag")
        where = (None, None, None, 0, None)
    else:
        _aux(pos, "pos", _F32, dev)
        _aux(tag, "tag", _U8, dev)
        if pos.dim() != 2 or pos.shape[1] != 3 or pos.shape[0] < n or tag.numel() < n:
            raise ValueError("pos must be [>= num_tokens, 3] and tag [>= num_tokens]")
        cu_ptr = frames_ptr = None
        if cu_requests is not None:
            _aux(cu_requests, "cu_requests", _I32, dev)
            nreq = cu_requests.numel() - 1
            cu_ptr = cu_requests.data_ptr()
        if start_frames is not None:
            _aux(start_frames, "start_frames", _F32, dev)
            if start_frames.numel() < max(nreq, 1):
                raise ValueError("start_frames must have one entry per request")
            frames_ptr = start_frames.data_ptr()
        where = (pos.data_ptr(), tag.data_ptr(), cu_ptr, nreq, frames_ptr)
    return where, (n, H, hk, D, 1 if kind is _BF16 else 0), q_stride, k_stride


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], q_weight: torch.Tensor,
                 k_weight: Optional[torch.Tensor], pos: Optional[torch.Tensor] = None,
                 tag: Optional[torch.Tensor] = None, cu_requests: Optional[torch.Tensor] = None,
                 start_frames: Optional[torch.Tensor] = None, num_tokens: Optional[int] = None,
                 eps: float = 1e-6, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, cfg: Optional[RopeConfig] = None):
    """RMS norm of every head's row of q [C, Hq, D] and k [C, Hk, D] (bf16) times q_weight / k_weight
    [D] (float32 or bfloat16), then the tagged RoPE of rope_apply; without pos and tag the norm alone.

    q and k may be parts of a fused projection (heads and dims contiguous, any token stride that is
    a multiple of 8); eps <= 0 selects 1e-6.  Writes new contiguous tensors unless q_out / k_out are
    given (q and k themselves are allowed); rows past num_tokens are left as they were.  Returns
    (q_out, k_out).
    """
    where, sizes, q_stride, k_stride = _norm_inputs(q, k, q_weight, k_weight, pos, tag, cu_requests, start_frames,
                                                    num_tokens)
    dev = q.device
    q_out_stride = k_out_stride = 0
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=_BF16, device=dev)
    else:
        q_out_stride = _rows(q_out, "q_out", dev, q.shape)
    if k is None:
        k_out = None
    elif k_out is None:
        k_out = torch.empty(k.shape, dtype=_BF16, device=dev)
    else:
        k_out_stride = _rows(k_out, "k_out", dev, k.shape)
    if sizes[0] == 0:
        return q_out, k_out
    desc = _QkNormDesc.pack(*sizes, eps, q_stride, k_stride, q_out_stride, k_out_stride, 0, 0)
    _launch(load_library().h3_qk_norm_rope, "h3_qk_norm_rope", dev, desc, q.data_ptr(), q_out.data_ptr(), _ptr(k),
            _ptr(k_out), q_weight.data_ptr(), k_weight.data_ptr() if k is not None else None, *where,
            ctypes.byref(cfg) if cfg is not None else None)
    return q_out, k_out


def qk_norm_rope_bwd_workspace_size(head_dim: int) -> int:
    return int(load_library().h3_qk_norm_rope_bwd_workspace_size(head_dim))


def qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: Optional[torch.Tensor], q: torch.Tensor,
                     k: Optional[torch.Tensor], q_weight: torch.Tensor, k_weight: Optional[torch.Tensor],
                     pos: Optional[torch.Tensor] = None, tag: Optional[torch.Tensor] = None,
                     cu_requests: Optional[torch.Tensor] = None,
                     start_frames: Optional[torch.Tensor] = None, num_tokens: Optional[int] = None,
                     eps: float = 1e-6, dq: Optional[torch.Tensor] = None,
                     dk: Optional[torch.Tensor] = None, cfg: Optional[RopeConfig] = None,
                     workspace: Optional[torch.Tensor] = None):
    """Gradient of qk_norm_rope: from dq_out, dk_out (bf16, the gradients of its outputs) and its
    inputs to (dq, dk bf16, dq_weight, dk_weight float32 [D]).  dq and dk may be parts of a fused
    gradient, or dq_out and dk_out, or q and k; the weights' gradients sum over tokens and heads in
    a fixed order.
    """
    where, sizes, q_stride, k_stride = _norm_inputs(q, k, q_weight, k_weight, pos, tag, cu_requests, start_frames,
                                                    num_tokens)
    dev, D, has_k = q.device, q.shape[2], k is not None
    dq_out_stride, dk_out_stride = _rows(dq_out, "dq_out", dev, q.shape), 0
    dq_stride = dk_stride = 0
    if dq is None:
        dq = torch.empty(q.shape, dtype=_BF16, device=dev)
    else:
        dq_stride = _rows(dq, "dq", dev, q.shape)
    dqw, dkw = torch.empty(D, dtype=_F32, device=dev), None
    if has_k:
        dk_out_stride = _rows(dk_out, "dk_out", dev, k.shape)
        if dk is None:
            dk = torch.empty(k.shape, dtype=_BF16, device=dev)
        else:
            dk_stride = _rows(dk, "dk", dev, k.shape)
        dkw = torch.empty(D, dtype=_F32, device=dev)
    else:
        dk = dk_out = None
    if sizes[0] == 0 and q.numel() == 0:  # no rows at all: no buffer to point at
        return dq, dk, dqw.zero_(), dkw.zero_() if has_k else None
    lib = load_library()
    if workspace is None:
        workspace = torch.empty(max(1, lib.h3_qk_norm_rope_bwd_workspace_size(D)), dtype=_U8, device=dev)
    else:
        _require(workspace, "workspace", _U8, dev)
    desc = _QkNormDesc.pack(*sizes, eps, q_stride, k_stride, dq_out_stride, dk_out_stride, dq_stride, dk_stride)
    _launch(lib.h3_qk_norm_rope_bwd, "h3_qk_norm_rope_bwd", dev, desc, dq_out.data_ptr(), _ptr(dk_out), q.data_ptr(),
            _ptr(k), q_weight.data_ptr(), k_weight.data_ptr() if has_k else None, *where,
            ctypes.byref(cfg) if cfg is not None else None, dq.data_ptr(), _ptr(dk), dqw.data_ptr(), _ptr(dkw),
            workspace.data_ptr(), workspace.numel())
    return dq, dk, dqw, dkw


_NORMS = {None: 0, "none": 0, "rms": 1, "layer": 2}
_TYPES = {torch.float32: 0, torch.bfloat16: 1}


class ResidualNormGrads(NamedTuple):
    """Gradients of residual_norm's inputs; None where the input is absent."""
    dx: torch.Tensor
    dy: Optional[torch.Tensor]
    weight: Optional[torch.Tensor]
    branch_weight: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    shift: Optional[torch.Tensor]
    gate: Optional[torch.Tensor]


def _like(t: torch.Tensor, dtype) -> torch.Tensor:
    """A new contiguous tensor of t's shape (empty_like is the cheaper call where it serves)."""
    if t.dtype is dtype and t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty(t.shape, dtype=dtype, device=t.device)


def _matrix(t: torch.Tensor, name: str, dtype, device: torch.device, shape=None) -> int:
    """Check [rows, dim] with contiguous rows; returns the row stride in elements, 0 when contiguous."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device and t.shape == shape:
        if t.is_contiguous():  # the common cases first
            return 0
        sr, sc = t.stride()
        if sc == 1 and sr >= shape[1] and shape[0] > 1:
            return sr
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be {'[rows, dim]' if shape is None else list(shape)}, got {list(t.shape)}")
    if t.is_contiguous():
        return 0
    sr, sc = t.stride()
    if sc != 1 or (t.shape[0] > 1 and sr < t.shape[1]):
        raise ValueError(f"{name} must have contiguous rows")
    return sr if t.shape[0] > 1 else 0


def _norm_kind(kind, name: str) -> int:
    if kind not in _NORMS:
        raise ValueError(f'{name} must be "rms", "layer" or "none"')
    return _NORMS[kind]


def _residual_norm_inputs(x, y, norm, weight, scale, shift, gate, branch_norm, branch_weight, residual_scale,
                          cu_requests, eps, num_tokens):
    """Checks shared by residual_norm and its backward; returns (sizes of the descriptor, row strides of
    x and y, strides of scale, shift and gate, pointers of the vectors and cu_requests)."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _TYPES:
        raise TypeError("the stream must be a float32 or bfloat16 tensor")
    dev = x.device
    x_stride, y_stride = _matrix(x, "x", x.dtype, dev), 0
    C, dim = x.shape
    n = C if num_tokens is None else int(num_tokens)
    if not 0 <= n <= C:
        raise ValueError("num_tokens must lie within the rows of x")
    kind, branch_kind = _norm_kind(norm, "norm"), _norm_kind(branch_norm, "branch_norm")
    if y is not None:
        y_stride = _matrix(y, "y", _BF16, dev, x.shape)
    elif branch_kind or gate is not None or branch_weight is not None or residual_scale != 1.0:
        raise ValueError("branch_norm, branch_weight, gate and residual_scale need y")
    if not kind and (y is None or weight is not None or scale is not None or shift is not None):
        raise ValueError('norm "none" leaves h out: it needs y, and takes no weight, scale or shift')
    requests, cu = 1, None
    if cu_requests is not None:
        _aux(cu_requests, "cu_requests", _I32, dev)
        requests = cu_requests.numel() - 1
        if requests < 1:
            raise ValueError("cu_requests must have one entry per request and one more")
        cu = cu_requests.data_ptr()
    weight_type = mod_type = None
    pointers, strides = [], []
    for name, t in (("weight", weight), ("branch_weight", branch_weight)):
        if t is None:
            pointers.append(None)
            continue
        if weight_type is None:
            weight_type = t.dtype if isinstance(t, torch.Tensor) else None
            if weight_type not in _TYPES:
                raise TypeError(f"{name} must be a float32 or bfloat16 tensor")
        _aux(t, name, weight_type, dev)
        if t.shape != (dim,):
            raise ValueError(f"{name} must be [dim]")
        pointers.append(t.data_ptr())
    for name, t in (("scale", scale), ("shift", shift), ("gate", gate)):
        if t is None:
            pointers.append(None)
            strides.append(0)
            continue
        if mod_type is None:
            mod_type = t.dtype if isinstance(t, torch.Tensor) else None
            if mod_type not in _TYPES:
                raise TypeError(f"{name} must be a float32 or bfloat16 tensor")
        strides.append(_matrix(t, name, mod_type, dev, (requests, dim)))
        pointers.append(t.data_ptr())
    pointers.append(cu)
    sizes = (n, dim, requests, kind, branch_kind, _TYPES[x.dtype], _TYPES.get(weight_type, 0), _TYPES.get(mod_type, 0),
             float(eps), float(residual_scale))
    return sizes, x_stride, y_stride, strides, pointers


def residual_norm(x: torch.Tensor, y: Optional[torch.Tensor] = None, norm: Optional[str] = "rms",
                  weight: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                  shift: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                  branch_norm: Optional[str] = None, branch_weight: Optional[torch.Tensor] = None,
                  residual_scale: float = 1.0, cu_requests: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  num_tokens: Optional[int] = None, x_out: Optional[torch.Tensor] = None,
                  h_out: Optional[torch.Tensor] = None):
    """The step between two branches of a block: the branch's output y joins the stream x, which is
    normed and modulated for the next branch.

      x' = residual_scale * x + gate * branch_norm(y) * branch_weight
      h  = norm(x') * weight * (1 + scale) + shift

    x float32 or bfloat16 [C, dim] (dim a multiple of 8, at most 8192), y bfloat16 [C, dim] or None (then
    x' is x); norm "rms", "layer" or "none" (no h), branch_norm the same ("none": y itself); weight,
    branch_weight [dim]; scale, shift, gate [R, dim], of the request that cu_requests (int32 [R+1], from 0 to
    num_tokens; None: one request) gives a token; each vector float32 or bfloat16, or None.  Rows may be
    parts of wider ones (a fused projection's six vectors, say).  Writes new tensors unless x_out / h_out are
    given (x and y themselves are allowed); rows past num_tokens are left as they were.  Returns (x', h),
    x' being x itself without y and h None with norm "none".
    """
    sizes, x_stride, y_stride, mod, ptr = _residual_norm_inputs(x, y, norm, weight, scale, shift, gate, branch_norm,
                                                                branch_weight, residual_scale, cu_requests, eps,
                                                                num_tokens)
    dev, x_out_stride, h_stride, h = x.device, 0, 0, None
    if y is None:
        if x_out is not None:
            raise ValueError("x_out needs y: without it the stream stays x")
        x_out = x
    elif x_out is None:
        x_out = _like(x, x.dtype)
    else:
        x_out_stride = _matrix(x_out, "x_out", x.dtype, dev, x.shape)
    if sizes[3]:
        if h_out is None:
            h = _like(x if y is None or x.dtype is _BF16 else y, _BF16)
        else:
            h, h_stride = h_out, _matrix(h_out, "h_out", _BF16, dev, x.shape)
    elif h_out is not None:
        raise ValueError('h_out needs a norm')
    if sizes[0] == 0:
        return x_out, h
    desc = _ResidualNormDesc.pack(*sizes, x_stride, y_stride, x_out_stride, h_stride, *mod, 0, 0, 0, 0)
    _launch(load_library().h3_residual_norm, "h3_residual_norm", dev, desc, x.data_ptr(), _ptr(y), *ptr,
            None if y is None else x_out.data_ptr(), _ptr(h))
    return x_out, h


def residual_norm_bwd_workspace_size(num_tokens: int, dim: int, num_requests: int = 1) -> int:
    desc = _ResidualNormDesc.pack(num_tokens, dim, num_requests, 0, 0, 0, 0, 0, 0.0, 1.0, *(0,) * 11)
    return int(load_library().h3_residual_norm_bwd_workspace_size(desc))


def residual_norm_bwd(dx_out: Optional[torch.Tensor], dh: Optional[torch.Tensor], x_out: torch.Tensor,
                      y: Optional[torch.Tensor] = None, norm: Optional[str] = "rms",
                      weight: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                      shift: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                      branch_norm: Optional[str] = None, branch_weight: Optional[torch.Tensor] = None,
                      residual_scale: float = 1.0, cu_requests: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      num_tokens: Optional[int] = None, dx: Optional[torch.Tensor] = None,
                      dy: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Gradient of residual_norm: from dx_out and dh, the gradients of its outputs (dx_out None: the stream
    is not used further), its output x_out (x itself without y) and its other inputs, to a
    ResidualNormGrads: dx in the stream's type, dy bfloat16, the vectors' in float32 (shift's values are not
    used: it says that its gradient is wanted).  dx may be dx_out or x_out, and dy y or dh; rows past
    num_tokens are left as they were and count for nothing.  Sums over tokens are taken in a fixed order.
    """
    sizes, x_stride, y_stride, mod, ptr = _residual_norm_inputs(x_out, y, norm, weight, scale, shift, gate, branch_norm,
                                                                branch_weight, residual_scale, cu_requests, eps,
                                                                num_tokens)
    dev, shape, has_y = x_out.device, x_out.shape, y is not None
    dx_out_stride = dh_stride = dx_stride = dy_stride = 0
    if dx_out is not None:
        dx_out_stride = _matrix(dx_out, "dx_out", x_out.dtype, dev, shape)
    elif not sizes[3]:
        raise ValueError('with norm "none" dx_out is the only gradient')
    if sizes[3]:
        dh_stride = _matrix(dh, "dh", _BF16, dev, shape)
    elif dh is not None:
        raise ValueError('dh needs a norm')
    if dx is None:
        dx = _like(x_out, x_out.dtype)
    else:
        dx_stride = _matrix(dx, "dx", x_out.dtype, dev, shape)
    if not has_y:
        if dy is not None:
            raise ValueError("dy needs y")
    elif dy is None:
        dy = _like(y, _BF16)
    else:
        dy_stride = _matrix(dy, "dy", _BF16, dev, shape)
    requests, dim = sizes[2], sizes[1]
    g = ResidualNormGrads(dx, dy, *(None if t is None else torch.empty(dim, dtype=_F32, device=dev)
                                    for t in (weight, branch_weight)),
                          *(None if t is None else torch.empty((requests, dim), dtype=_F32, device=dev)
                            for t in (scale, shift, gate)))
    if x_out.numel() == 0:  # no rows at all: no buffer to point at
        for t in g[2:]:
            if t is not None:
                t.zero_()
        return g
    lib = load_library()
    desc = _ResidualNormDesc.pack(*sizes, 0, y_stride, x_stride, 0, *mod, dx_out_stride, dh_stride, dx_stride, dy_stride)
    if workspace is None:
        workspace = torch.empty(lib.h3_residual_norm_bwd_workspace_size(desc) or 1, dtype=_U8, device=dev)
    else:
        _require(workspace, "workspace", _U8, dev)
    _launch(lib.h3_residual_norm_bwd, "h3_residual_norm_bwd", dev, desc, _ptr(dx_out), _ptr(dh), x_out.data_ptr(),
            _ptr(y), ptr[0], ptr[1], ptr[2], ptr[4], ptr[5], dx.data_ptr(), _ptr(dy), _ptr(g.weight),
            _ptr(g.branch_weight), _ptr(g.scale), _ptr(g.shift), _ptr(g.gate), workspace.data_ptr(),
            workspace.numel())
    return g


_E4M3 = torch.float8_e4m3fn


def _cache_inputs(k_cache, v_cache, k_scale, v_scale, block_table, segments, dev):
    """Checks of a paged cache; returns (heads, head_dim, type, page_size, num_pages, max_pages) and its pointers."""
    kind = k_cache.dtype if isinstance(k_cache, torch.Tensor) else None
    if kind is not _BF16 and kind is not _E4M3:
        raise TypeError("k_cache must be a bfloat16 or float8_e4m3fn tensor")
    _aux(k_cache, "k_cache", kind, dev)
    _aux(v_cache, "v_cache", kind, dev)
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [num_pages, num_heads, page_size, head_dim]")
    scales = None, None
    if kind is _E4M3:
        if k_scale is None or v_scale is None:
            raise ValueError("an e4m3 cache needs k_scale and v_scale")
        _aux(k_scale, "k_scale", _U8, dev)
        _aux(v_scale, "v_scale", _U8, dev)
        if k_scale.shape != shape[:3] or v_scale.shape != shape[:3]:
            raise ValueError("k_scale and v_scale must be [num_pages, num_heads, page_size]")
        scales = k_scale.data_ptr(), v_scale.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise ValueError("a bfloat16 cache takes no scales")
    _aux(block_table, "block_table", _I32, dev)
    if block_table.dim() != 2 or block_table.shape[0] != segments:
        raise ValueError("block_table must be [num_segments, max_pages]")
    return (shape[1], shape[3], 1 if kind is _BF16 else 2, shape[2], shape[0], block_table.shape[1]), \
        (k_cache.data_ptr(), v_cache.data_ptr(), *scales, block_table.data_ptr())


def _cache_call(name, rows, strides, k_cache, v_cache, block_table, cu_seqlens, start, k_scale, v_scale, write):
    dev = k_cache.device
    _aux(cu_seqlens, "cu_seqlens", _I32, dev)
    _aux(start, "start", _I32, dev)
    S = cu_seqlens.numel() - 1
    if S < 0 or start.numel() != S:
        raise ValueError("cu_seqlens must have one entry per segment and one more, start one per segment")
    (heads, dim, *rest), pointers = _cache_inputs(k_cache, v_cache, k_scale, v_scale, block_table, S, dev)
    C = rows[0].shape[0]
    if rows[0].shape[1:] != (heads, dim):
        raise ValueError("k and v must be [C, num_heads, head_dim] of the cache's heads")
    if C == 0 or S == 0:
        return
    desc = _KvCacheDesc.pack(S, C, heads, dim, *rest, *strides)
    kv, where = tuple(t.data_ptr() for t in rows), (*pointers, cu_seqlens.data_ptr(), start.data_ptr())
    _launch(getattr(load_library(), name), name, dev, desc, *(kv + where if write else where + kv))


def kv_cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_table: torch.Tensor, cu_seqlens: torch.Tensor, start: torch.Tensor,
                   k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None) -> None:
    """Row i of segment g (row cu_seqlens[g] + i of k and v, bf16 [C, H, D]) into a paged cache at position
    start[g] + i of the segment: page block_table[g, position // page_size], row position % page_size.

    k_cache, v_cache [num_pages, H, page_size, D], page_size 16, 32, 64, 128 or 256: bfloat16, or
    float8_e4m3fn with k_scale, v_scale uint8 [num_pages, H, page_size], which hold e + 127 for the row's scale
    2^e, the least with which its largest value fits e4m3.  block_table int32 [S, max_pages], cu_seqlens
    int32 [S+1], start int32 [S].  k and v may be parts of a fused projection.
    """
    strides = _rows(k, "k", k_cache.device), _rows(v, "v", k_cache.device, k.shape)
    _cache_call("h3_kv_cache_write", (k, v), strides, k_cache, v_cache, block_table, cu_seqlens, start, k_scale,
                v_scale, True)


def kv_cache_read(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                  cu_seqlens: torch.Tensor, start: torch.Tensor, num_rows: Optional[int] = None,
                  k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                  k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None):
    """The reverse of kv_cache_write: positions start[g] + i into row cu_seqlens[g] + i of k and v (bf16
    [C, H, D]), the values that the cache holds.  New tensors of num_rows rows unless k_out and v_out are
    given; rows past the last segment are left as they were.  Returns (k, v)."""
    dev = k_cache.device
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages, num_heads, page_size, head_dim]")
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out are given together")
    if k_out is None:
        if num_rows is None:
            raise ValueError("num_rows or k_out and v_out are needed")
        shape = (int(num_rows), k_cache.shape[1], k_cache.shape[3])
        k_out, v_out = (torch.empty(shape, dtype=_BF16, device=dev) for _ in range(2))
        strides = 0, 0
    else:
        strides = _rows(k_out, "k_out", dev), _rows(v_out, "v_out", dev, k_out.shape)
    _cache_call("h3_kv_cache_read", (k_out, v_out), strides, k_cache, v_cache, block_table, cu_seqlens, start, k_scale,
                v_scale, False)
    return k_out, v_out


def paged_attn_workspace_size(num_segments: int, max_seqlen_q: int, max_seqlen_k: int, capacity_q: int,
                              num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int = 16,
                              e4m3: bool = False, max_pages: Optional[int] = None) -> int:
    """Bytes for paged_attn_fwd's workspace; max_pages: the block table's width (None: what max_seqlen_k needs).
    For long chunks over an e4m3 cache they include room for its tokens in bf16; without it (the size with
    e4m3=False) the call gives the same and takes longer."""
    pages = -(-max_seqlen_k // page_size) if max_pages is None else max_pages
    desc = _PagedAttnDesc.pack(num_segments, max_seqlen_q, max_seqlen_k, capacity_q, num_q_heads, num_kv_heads,
                               head_dim, 2 if e4m3 else 1, page_size, 1, pages, 0, 0.0, 0)
    return int(load_library().h3_paged_attn_workspace_size(desc))


def _paged_workspace(lib, desc: bytes, e4m3: bool, limit: Optional[int], dev: torch.device) -> torch.Tensor:
    """A workspace for the call: with room for unpacking where the limit and the device's memory allow it."""
    size = lib.h3_paged_attn_workspace_size(desc) or 16
    if not e4m3:
        return torch.empty(size, dtype=_U8, device=dev)
    if limit is None or size <= limit:
        try:
            return torch.empty(size, dtype=_U8, device=dev)
        except torch.OutOfMemoryError:
            pass
    plain = _PagedAttnDesc.from_buffer_copy(desc)
    plain.cache_type = 1  # what a bf16 cache wants is the least
    return torch.empty(lib.h3_paged_attn_workspace_size(bytes(plain)) or 16, dtype=_U8, device=dev)


def paged_attn_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                   cu_seqlens_q: torch.Tensor, seqused_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int,
                   k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                   causal_block: int = 0, out: Optional[torch.Tensor] = None, return_lse: bool = False,
                   lse: Optional[torch.Tensor] = None, softmax_scale: Optional[float] = None,
                   workspace: Optional[torch.Tensor] = None, workspace_limit: Optional[int] = None):
    """Attention of new tokens over a paged cache: the query rows of segment g (cu_seqlens_q, int32 [S+1]) are
    the last of its seqused_k[g] cached tokens (int32 [S]), whose keys and values kv_cache_write has put
    into k_cache, v_cache (and k_scale, v_scale) under block_table.

    q bf16 [C, Hq, D], Hkv dividing Hq; may be a part of a fused projection.  causal_block 0: every row sees
    every cached token; B > 0: the row at position p of its sequence sees those before (p // B + 1) * B, so
    1 is causal by token and the tokens of a frame causal by frame.  max_seqlen_q and max_seqlen_k bound a
    segment's rows and tokens; when max_seqlen_q * Hq / Hkv is at most 16 the cache is streamed once for all
    of a key head's rows, so single tokens want a tight bound.  A row that sees nothing gives 0 and an
    LSE of -inf; rows of `out` outside every segment are left untouched.  Returns out [C, Hq, D] (and lse
    fp32 [Hq, C] when requested).

    Long chunks (max_seqlen_q * Hq / Hkv above 512) over an e4m3 cache are fastest with its tokens unpacked to
    bf16 in the workspace: twice the e4m3 bytes of S * max_seqlen_k tokens, so tight bounds save memory.  Where
    that is more than 4 GiB, or workspace_limit bytes (None: no limit) or the device's free memory do not hold it, the
    call allocates the least workspace instead, gives the same results and takes longer.
    """
    dev = q.device
    q_stride = _rows(q, "q", dev)
    C, H, D = q.shape
    _aux(cu_seqlens_q, "cu_seqlens_q", _I32, dev)
    _aux(seqused_k, "seqused_k", _I32, dev)
    S = cu_seqlens_q.numel() - 1
    if S < 0 or seqused_k.numel() != S:
        raise ValueError("cu_seqlens_q must have one entry per segment and one more, seqused_k one per segment")
    (heads, dim, *rest), cache = _cache_inputs(k_cache, v_cache, k_scale, v_scale, block_table, S, dev)
    if dim != D:
        raise ValueError("the cache must have q's head_dim")
    if out is None:
        out = _like(q, _BF16)
    else:
        _require(out, "out", _BF16, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if lse is not None:
        _require(lse, "lse", _F32, dev)
        if lse.shape != (H, C):
            raise ValueError("lse must be [Hq, C]")
    elif return_lse:
        lse = torch.empty((H, C), dtype=_F32, device=dev)
    if C > 0:
        lib = load_library()
        desc = _PagedAttnDesc.pack(S, int(max_seqlen_q), int(max_seqlen_k), C, H, heads, D, *rest, int(causal_block),
                                   0.0 if softmax_scale is None else float(softmax_scale), q_stride)
        if workspace is None:
            workspace = _paged_workspace(lib, desc, e4m3=rest[0] == 2, limit=workspace_limit, dev=dev)
        else:
            _require(workspace, "workspace", _U8, dev)
        _launch(lib.h3_paged_attn_fwd, "h3_paged_attn_fwd", dev, desc, q.data_ptr(), *cache, cu_seqlens_q.data_ptr(),
                seqused_k.data_ptr(), out.data_ptr(), _ptr(lse), workspace.data_ptr(), workspace.numel())
    return (out, lse) if lse is not None else out


def varlen_attn_workspace_size(num_segments: int, num_heads: int, max_seqlen: int, head_dim: int) -> int:
    return int(load_library().h3_varlen_attn_workspace_size(num_segments, num_heads, max_seqlen, head_dim))


def varlen_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                    max_seqlen: int, out: Optional[torch.Tensor] = None, return_lse: bool = False,
                    lse: Optional[torch.Tensor] = None, softmax_scale: Optional[float] = None,
                    workspace: Optional[torch.Tensor] = None):
    """Block-diagonal attention over the segments of cu_seqlens (int32 [S+1], device).

    q, k, v: bf16 [C, H, D] with C >= cu_seqlens[-1].  Rows of `out` outside every segment are
    left untouched.  Returns out (and lse fp32 [H, C] when requested).  For segments of a few hundred to a
    few thousand rows varlen_cross_attn_fwd with equal offsets is the faster form.
    """
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v)):
        _require(t, name, torch.bfloat16, dev)
    if q.dim() != 3 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must all be [C, H, D]")
    C, H, D = q.shape
    _require(cu_seqlens, "cu_seqlens", torch.int32, dev)
    S = cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty_like(q)
    _require(out, "out", torch.bfloat16, dev)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if return_lse and lse is None:
        lse = torch.empty((H, C), dtype=torch.float32, device=dev)
    if lse is not None:
        _require(lse, "lse", torch.float32, dev)
        if tuple(lse.shape) != (H, C):
            raise ValueError("lse must be [H, C]")
    lib = load_library()
    ws_need = int(lib.h3_varlen_attn_workspace_size(S, H, int(max_seqlen), D))
    if ws_need > 0 and workspace is None:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=dev)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    scale = 0.0 if softmax_scale is None else float(softmax_scale)
    with torch.cuda.device(dev):
        st = lib.h3_varlen_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                    _ptr(cu_seqlens), S, int(max_seqlen), C, H, D, scale,
                                    _ptr(workspace), ws_bytes, _stream(dev))
    _check(st, "h3_varlen_attn_fwd")
    return (out, lse) if (return_lse or lse is not None) else out


def varlen_attn_fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                            cu_seqlens: torch.Tensor, max_seqlen: int, out: torch.Tensor,
                            lse: Optional[torch.Tensor] = None,
                            softmax_scale: Optional[float] = None) -> torch.Tensor:
    """varlen_attn_fwd through the entry point that allocates no device memory.

    For callers that cannot allocate: `out` (and `lse`, if wanted) must be given, and the
    library uses its own fixed scratch array (at most 16384 segments).  Calls on one device must
    not overlap on the GPU; the first call on a device should come before any stream capture.
    """
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        _require(t, name, torch.bfloat16, dev)
    if q.dim() != 3 or k.shape != q.shape or v.shape != q.shape or out.shape != q.shape:
        raise ValueError("q, k, v, out must all be [C, H, D]")
    C, H, D = q.shape
    _require(cu_seqlens, "cu_seqlens", torch.int32, dev)
    if lse is not None:
        _require(lse, "lse", torch.float32, dev)
        if tuple(lse.shape) != (H, C):
            raise ValueError("lse must be [H, C]")
    scale = 0.0 if softmax_scale is None else float(softmax_scale)
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.h3_varlen_attn_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                            _ptr(cu_seqlens), cu_seqlens.numel() - 1,
                                            int(max_seqlen), C, H, D, scale, _stream(dev))
    _check(st, "h3_varlen_attn_fwd_noalloc")
    return out


def _cross_inputs(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, seqused_k, softmax_scale):
    """Checks shared by the cross attention calls; returns the descriptor's values and the offsets'
    pointers."""
    dev = q.device
    q_stride, k_stride = _rows(q, "q", dev), _rows(k, "k", dev)
    v_stride = _rows(v, "v", dev, k.shape)
    C, H, D = q.shape
    Ck, Hk, Dk = k.shape
    if Dk != D:
        raise ValueError("k and v must have q's head_dim")
    _aux(cu_seqlens_q, "cu_seqlens_q", _I32, dev)
    _aux(cu_seqlens_k, "cu_seqlens_k", _I32, dev)
    S = cu_seqlens_q.numel() - 1
    if S < 0 or cu_seqlens_k.numel() != S + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have one entry per segment and one more")
    used = None
    if seqused_k is not None:
        _aux(seqused_k, "seqused_k", _I32, dev)
        if seqused_k.numel() != S:
            raise ValueError("seqused_k must have one entry per segment")
        used = seqused_k.data_ptr()
    sizes = (S, int(max_seqlen_q), int(max_seqlen_k), C, Ck, H, Hk, D,
             0.0 if softmax_scale is None else float(softmax_scale), q_stride, k_stride, v_stride)
    return sizes, (cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), used)


def varlen_cross_attn_workspace_size(num_segments: int, max_seqlen_q: int, max_seqlen_k: int, capacity_q: int,
                                     capacity_k: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    desc = _CrossAttnDesc.pack(num_segments, max_seqlen_q, max_seqlen_k, capacity_q, capacity_k, num_q_heads,
                               num_kv_heads, head_dim, 0.0, 0, 0, 0, 0, 0, 0)
    return int(load_library().h3_varlen_cross_attn_workspace_size(desc))


def varlen_cross_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens_q: torch.Tensor,
                          cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int,
                          seqused_k: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                          return_lse: bool = False, lse: Optional[torch.Tensor] = None,
                          softmax_scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None):
    """Packed cross attention: the query rows of segment g (cu_seqlens_q, int32 [S+1]) attend to the key
    rows of segment g (cu_seqlens_k, int32 [S+1]; its first seqused_k[g] rows when given).

    q bf16 [Cq, Hq, D]; k, v bf16 [Ck, Hkv, D] with Hkv dividing Hq; each may be a part of a fused
    projection (heads and dims contiguous, any token stride that is a multiple of 8).  max_seqlen_q
    and max_seqlen_k bound a segment's rows and used keys; when max_seqlen_q * Hq / Hkv is at most 16 the keys
    are read once for all of a key head's rows, so single tokens want a tight bound.  A segment without keys
    gives 0 and an LSE of -inf; rows of `out` outside every segment are left untouched.  Returns out [Cq, Hq, D] (and lse
    fp32 [Hq, Cq] when requested).
    """
    sizes, offsets = _cross_inputs(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, seqused_k,
                                   softmax_scale)
    dev = q.device
    C, H = sizes[3], sizes[5]
    if out is None:
        out = torch.empty(q.shape, dtype=_BF16, device=dev)
    else:
        _require(out, "out", _BF16, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if lse is not None:
        _require(lse, "lse", _F32, dev)
        if lse.shape != (H, C):
            raise ValueError("lse must be [Hq, Cq]")
    elif return_lse:
        lse = torch.empty((H, C), dtype=_F32, device=dev)
    if C > 0:
        lib = load_library()
        desc = _CrossAttnDesc.pack(*sizes, 0, 0, 0)
        if workspace is None:
            need = lib.h3_varlen_cross_attn_workspace_size(desc)
            workspace = torch.empty(need or 1, dtype=_U8, device=dev)
        else:
            _require(workspace, "workspace", _U8, dev)
        _launch(lib.h3_varlen_cross_attn_fwd, "h3_varlen_cross_attn_fwd", dev, desc, q.data_ptr(), k.data_ptr(),
                v.data_ptr(), out.data_ptr(), _ptr(lse), *offsets, workspace.data_ptr(), workspace.numel())
    return (out, lse) if lse is not None else out


def varlen_cross_attn_bwd_workspace_size(num_segments: int, max_seqlen_q: int, max_seqlen_k: int, capacity_q: int,
                                         capacity_k: int, num_q_heads: int, num_kv_heads: int,
                                         head_dim: int) -> int:
    desc = _CrossAttnDesc.pack(num_segments, max_seqlen_q, max_seqlen_k, capacity_q, capacity_k, num_q_heads,
                               num_kv_heads, head_dim, 0.0, 0, 0, 0, 0, 0, 0)
    return int(load_library().h3_varlen_cross_attn_bwd_workspace_size(desc))


def varlen_cross_attn_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                          out: torch.Tensor, lse: torch.Tensor, cu_seqlens_q: torch.Tensor,
                          cu_seqlens_k: torch.Tensor, max_seqlen_q: int, max_seqlen_k: int,
                          seqused_k: Optional[torch.Tensor] = None, dq: Optional[torch.Tensor] = None,
                          dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
                          softmax_scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None):
    """Gradient of varlen_cross_attn_fwd (with equal offsets, of varlen_attn_fwd): from dout (the gradient
    of its output), its inputs, its output and its LSE to (dq, dk, dv), bf16, shaped as q, k, v.

    dq, dk and dv may be parts of a fused gradient.  Every row of every segment is written (0 for keys
    that a segment does not use); other rows are left untouched.  The result does not depend on timing.
    """
    sizes, offsets = _cross_inputs(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, seqused_k,
                                   softmax_scale)
    dev, shape, kshape = q.device, q.shape, k.shape
    for name, t in (("dout", dout), ("out", out)):
        _aux(t, name, _BF16, dev)
        if t.shape != shape:
            raise ValueError(f"{name} must have q's shape")
    _aux(lse, "lse", _F32, dev)
    if lse.shape != (sizes[5], sizes[3]):
        raise ValueError("lse must be [Hq, Cq]")
    strides = [0, 0, 0]
    if dq is None:
        dq = torch.empty(shape, dtype=_BF16, device=dev)
    else:
        strides[0] = _rows(dq, "dq", dev, shape)
    if dk is None:
        dk = torch.empty(kshape, dtype=_BF16, device=dev)
    else:
        strides[1] = _rows(dk, "dk", dev, kshape)
    if dv is None:
        dv = torch.empty(kshape, dtype=_BF16, device=dev)
    else:
        strides[2] = _rows(dv, "dv", dev, kshape)
    lib = load_library()
    desc = _CrossAttnDesc.pack(*sizes, *strides)
    if workspace is None:
        need = lib.h3_varlen_cross_attn_bwd_workspace_size(desc)
        workspace = torch.empty(need or 1, dtype=_U8, device=dev)
    else:
        _require(workspace, "workspace", _U8, dev)
    _launch(lib.h3_varlen_cross_attn_bwd, "h3_varlen_cross_attn_bwd", dev, desc, dout.data_ptr(), q.data_ptr(),
            k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), *offsets, dq.data_ptr(), dk.data_ptr(),
            dv.data_ptr(), workspace.data_ptr(), workspace.numel())
    return dq, dk, dv


def window_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, grid: Sequence[int],
                    win: Sequence[int], shift: Sequence[int], out: Optional[torch.Tensor] = None,
                    return_lse: bool = False, lse: Optional[torch.Tensor] = None,
                    softmax_scale: Optional[float] = None):
    """Shifted 3D window attention in place on the grid (no packed copies).

    q, k, v: bf16 [T*H*W, heads, D] in row-major (t, h, w) token order.  Returns out (and lse
    fp32 [heads, T*H*W] when requested), in the same order.
    """
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v)):
        _require(t, name, torch.bfloat16, dev)
    n = int(grid[0]) * int(grid[1]) * int(grid[2])
    if q.dim() != 3 or q.shape[0] != n or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must be [T*H*W, heads, D]")
    _, H, D = q.shape
    out = torch.empty_like(q) if out is None else out
    _require(out, "out", torch.bfloat16, dev)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if return_lse and lse is None:
        lse = torch.empty((H, n), dtype=torch.float32, device=dev)
    if lse is not None:
        _require(lse, "lse", torch.float32, dev)
        if tuple(lse.shape) != (H, n):
            raise ValueError("lse must be [heads, T*H*W]")
    scale = 0.0 if softmax_scale is None else float(softmax_scale)
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.h3_window_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _i3(grid),
                                    _i3(win), _i3(shift), H, D, scale, _stream(dev))
    _check(st, "h3_window_attn_fwd")
    return (out, lse) if (return_lse or lse is not None) else out


def window_count(grid: Sequence[int], win: Sequence[int], shift: Sequence[int]) -> int:
    n = load_library().h3_window_count(_i3(grid), _i3(win), _i3(shift))
    if n < 0:
        raise ValueError("invalid window geometry")
    return int(n)


def window_pack(grid: Sequence[int], win: Sequence[int], shift: Sequence[int],
                tensors: Sequence[torch.Tensor] = (), device: Optional[torch.device] = None,
                perm: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                outs: Optional[Sequence[torch.Tensor]] = None):
    """Partition the (T, H, W) grid into (shifted) windows and gather each tensor's rows.

    tensors: [N, ...] contiguous, same device, N = T*H*W.  Returns (perm, cu_seqlens, packed).
    """
    nwin = window_count(grid, win, shift)
    n = int(grid[0]) * int(grid[1]) * int(grid[2])
    dev = tensors[0].device if tensors else (device or torch.device("cuda"))
    if perm is None:
        perm = torch.empty(n, dtype=torch.int32, device=dev)
    if cu_seqlens is None:
        cu_seqlens = torch.empty(nwin + 1, dtype=torch.int32, device=dev)
    _require(perm, "perm", torch.int32, dev)
    _require(cu_seqlens, "cu_seqlens", torch.int32, dev)
    if perm.numel() < n or cu_seqlens.numel() < nwin + 1:
        raise ValueError("perm / cu_seqlens too small")
    outs = list(outs) if outs is not None else [torch.empty_like(t) for t in tensors]
    row_bytes = 0
    for i, (t, o) in enumerate(zip(tensors, outs)):
        if not t.is_contiguous() or not o.is_contiguous() or t.device != dev or o.device != dev:
            raise ValueError("window_pack tensors must be contiguous on one device")
        if t.shape[0] != n or o.shape != t.shape or o.dtype != t.dtype:
            raise ValueError("each tensor must have T*H*W rows and a matching output")
        rb = t[0].numel() * t.element_size()
        if i and rb != row_bytes:
            raise ValueError("all tensors must share one row size")
        row_bytes = rb
    k = len(tensors)
    src = (ctypes.c_void_p * max(k, 1))(*[t.data_ptr() for t in tensors])
    dst = (ctypes.c_void_p * max(k, 1))(*[o.data_ptr() for o in outs])
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.h3_window_pack(_i3(grid), _i3(win), _i3(shift), _ptr(perm), _ptr(cu_seqlens),
                                src, dst, k, row_bytes, _stream(dev))
    _check(st, "h3_window_pack")
    return perm, cu_seqlens, outs


def window_unpack(perm: torch.Tensor, src: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Restore original order: out[perm[j]] = src[j]."""
    dev = src.device
    _require(perm, "perm", torch.int32, dev)
    if not src.is_contiguous():
        raise ValueError("src must be contiguous")
    n = src.shape[0]
    if perm.numel() < n:
        raise ValueError("perm too small")
    out = torch.empty_like(src) if out is None else out
    if out.shape != src.shape or out.dtype != src.dtype or not out.is_contiguous():
        raise ValueError("out must match src")
    row_bytes = src[0].numel() * src.element_size()
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.h3_window_unpack(_ptr(perm), n, _ptr(src), _ptr(out), row_bytes, _stream(dev))
    _check(st, "h3_window_unpack")
    return out


def vsa_block_count(grid: Sequence[int], block: Sequence[int] = (4, 4, 4)) -> int:
    n = load_library().h3_vsa_block_count(_i3(grid), _i3(block))
    if n < 0:
        raise ValueError("invalid VSA block geometry")
    return int(n)


def vsa_select_workspace_size(grid: Sequence[int], block: Sequence[int], num_heads: int,
                              head_dim: int) -> int:
    return int(load_library().h3_vsa_select_workspace_size(_i3(grid), _i3(block), num_heads, head_dim))


def vsa_select(q: torch.Tensor, k: torch.Tensor, grid: Sequence[int], topk: int,
               block: Sequence[int] = (4, 4, 4), scores: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               softmax_scale: Optional[float] = None):
    """Block gate scores and top-k key blocks per query block (VSA).

    q, k: bf16 [T*H*W, heads, D] in row-major (t, h, w) order.  Returns (block_idx int32
    [heads, nblk, topk] in ascending block id, scores fp32 [heads, nblk, nblk]).
    """
    dev = q.device
    _require(q, "q", torch.bfloat16, dev)
    _require(k, "k", torch.bfloat16, dev)
    n = int(grid[0]) * int(grid[1]) * int(grid[2])
    if q.dim() != 3 or q.shape[0] != n or k.shape != q.shape:
        raise ValueError("q, k must be [T*H*W, heads, D]")
    _, H, D = q.shape
    nblk = vsa_block_count(grid, block)
    if scores is None:
        scores = torch.empty((H, nblk, nblk), dtype=torch.float32, device=dev)
    if out is None:
        out = torch.empty((H, nblk, int(topk)), dtype=torch.int32, device=dev)
    _require(scores, "scores", torch.float32, dev)
    _require(out, "out", torch.int32, dev)
    if tuple(scores.shape) != (H, nblk, nblk) or tuple(out.shape) != (H, nblk, int(topk)):
        raise ValueError("scores must be [heads, nblk, nblk] and out [heads, nblk, topk]")
    need = vsa_select_workspace_size(grid, block, H, D)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _require(workspace, "workspace", torch.uint8, dev)
    scale = 0.0 if softmax_scale is None else float(softmax_scale)
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.h3_vsa_select(_ptr(q), _ptr(k), _i3(grid), _i3(block), H, D, int(topk), scale,
                               _ptr(scores), _ptr(out), _ptr(workspace), workspace.numel(),
                               _stream(dev))
    _check(st, "h3_vsa_select")
    return out, scores


def vsa_attn_workspace_size(grid: Sequence[int], block: Sequence[int], num_heads: int,
                            topk: int) -> int:
    return int(load_library().h3_vsa_attn_workspace_size(_i3(grid), _i3(block), num_heads, topk))


def vsa_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, grid: Sequence[int],
                 block_idx: torch.Tensor, block: Sequence[int] = (4, 4, 4),
                 out: Optional[torch.Tensor] = None, return_lse: bool = False,
                 lse: Optional[torch.Tensor] = None, softmax_scale: Optional[float] = None,
                 workspace: Optional[torch.Tensor] = None):
    """Token-level attention of every query block over its selected key blocks (VSA).

    q, k, v: bf16 [T*H*W, heads, D] in row-major (t, h, w) order; block_idx int32
    [heads, nblk, topk]; workspace uint8 of vsa_attn_workspace_size() bytes (allocated when
    omitted).  Returns out (and lse fp32 [heads, T*H*W] when requested).
    """
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v)):
        _require(t, name, torch.bfloat16, dev)
    n = int(grid[0]) * int(grid[1]) * int(grid[2])
    if q.dim() != 3 or q.shape[0] != n or k.shape != q.shape or v.shape != q.shape:
        raise ValueError("q, k, v must be [T*H*W, heads, D]")
    _, H, D = q.shape
    nblk = vsa_block_count(grid, block)
    _require(block_idx, "block_idx", torch.int32, dev)
    if block_idx.dim() != 3 or tuple(block_idx.shape[:2]) != (H, nblk):
        raise ValueError("block_idx must be [heads, nblk, topk]")
    topk = int(block_idx.shape[2])
    out = torch.empty_like(q) if out is None else out
    _require(out, "out", torch.bfloat16, dev)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if return_lse and lse is None:
        lse = torch.empty((H, n), dtype=torch.float32, device=dev)
    if lse is not None:
        _require(lse, "lse", torch.float32, dev)
        if tuple(lse.shape) != (H, n):
            raise ValueError("lse must be [heads, T*H*W]")
    scale = 0.0 if softmax_scale is None else float(softmax_scale)
    need = vsa_attn_workspace_size(grid, block, H, topk)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _require(workspace, "workspace", torch.uint8, dev)
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.h3_vsa_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _i3(grid),
                                 _i3(block), H, D, _ptr(block_idx), topk, scale, _ptr(workspace),
                                 workspace.numel(), _stream(dev))
    _check(st, "h3_vsa_attn_fwd")
    return (out, lse) if (return_lse or lse is not None) else out


def continuation_config(text_rows: int, clip_video_frames: int, clip_audio_rows: int, frame_h: int,
                        frame_w: int, new_video_frames: int, new_audio_rows: int, tail_frames: int = 7,
                        frames_per_latent: int = 4) -> ContinuationConfig:
    return ContinuationConfig(text_rows, clip_video_frames, clip_audio_rows, frame_h, frame_w,
                              new_video_frames, new_audio_rows, tail_frames, frames_per_latent)


def continuation_plan(cfg: ContinuationConfig) -> ContinuationPlan:
    """Index math of a continuation window (host only)."""
    plan = ContinuationPlan()
    _check(load_library().h3_continuation_make_plan(ctypes.byref(cfg), ctypes.byref(plan)),
           "h3_continuation_make_plan")
    return plan


def _rows2d(t: Optional[torch.Tensor], name: str):
    if t is None:
        return None, 0
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t, t[0].numel() * t.element_size() if t.shape[0] > 0 else 0


def continuation_pack(cfg: ContinuationConfig, text, clip_video, clip_audio, new_video, new_audio,
                      out: Optional[torch.Tensor] = None):
    """The five-group DiT sequence of a continuation window: returns (rows, pos fp32 [N, 3],
    tag u8 [N], target u8 [N]).  Row tensors are [n, ...] with one common row size."""
    plan = continuation_plan(cfg)
    srcs = [text, clip_video, clip_audio, new_video, new_audio]
    ref = next(t for t in srcs if t is not None and t.shape[0] > 0)
    dev = ref.device
    row_bytes = ref[0].numel() * ref.element_size()
    for i, t in enumerate(srcs):
        if t is not None and t.shape[0] > 0:
            _, rb = _rows2d(t, f"source {i}")
            if rb != row_bytes or t.dtype != ref.dtype:
                raise ValueError("all row tensors need the same row size and dtype")
    n = plan.num_rows
    out = torch.empty((n,) + tuple(ref.shape[1:]), dtype=ref.dtype, device=dev) if out is None else out
    pos = torch.empty((n, 3), dtype=torch.float32, device=dev)
    tag = torch.empty(n, dtype=torch.uint8, device=dev)
    target = torch.empty(n, dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        st = load_library().h3_continuation_pack(ctypes.byref(cfg), _ptr(text), _ptr(clip_video),
                                                 _ptr(clip_audio), _ptr(new_video), _ptr(new_audio),
                                                 row_bytes, _ptr(out), _ptr(pos), _ptr(tag), _ptr(target),
                                                 _stream(dev))
    _check(st, "h3_continuation_pack")
    return out, pos, tag, target


def continuation_append(cfg: ContinuationConfig, new_video: torch.Tensor, new_audio: torch.Tensor,
                        clip_video: torch.Tensor, clip_audio: torch.Tensor):
    """Append the new window's rows past the overlap to the clip buffers (in place; they must
    have room for the plan's out_video_frames / out_audio_rows).  Returns the plan."""
    plan = continuation_plan(cfg)
    ref = new_video if new_video.shape[0] > 0 else new_audio
    row_bytes = ref[0].numel() * ref.element_size()
    dev = ref.device
    hw = cfg.frame_h * cfg.frame_w
    with torch.cuda.device(dev):
        st = load_library().h3_continuation_append(ctypes.byref(cfg), _ptr(new_video), _ptr(new_audio),
                                                   row_bytes, _ptr(clip_video), clip_video.shape[0],
                                                   _ptr(clip_audio), clip_audio.shape[0], _stream(dev))
    _check(st, "h3_continuation_append")
    assert plan.out_video_frames * hw <= clip_video.shape[0]
    return plan


def masked_row_update(dst: torch.Tensor, src: torch.Tensor, mask: torch.Tensor) -> torch.Tensor:
    """dst[i] = src[i] where mask[i] (uint8) is non-zero; in place on dst."""
    if dst.shape != src.shape or dst.dtype != src.dtype or mask.dtype != torch.uint8:
        raise ValueError("dst and src must match; mask must be uint8")
    n = dst.shape[0]
    row_bytes = dst[0].numel() * dst.element_size() if n > 0 else 16
    with torch.cuda.device(dst.device):
        st = load_library().h3_masked_row_update(_ptr(dst), _ptr(src), _ptr(mask), n, row_bytes,
                                                 _stream(dst.device))
    _check(st, "h3_masked_row_update")
    return dst


def _np_ptr(a):
    return ctypes.c_void_p(a.ctypes.data) if a is not None and a.size else None


def sp_assign_windows(grid: Sequence[int], win: Sequence[int], shift: Sequence[int], world: int):
    """Owner rank of every window of one layer (longest-first on token counts) and the tokens
    each rank owns: (window_rank int32 [nwin], rank_tokens int64 [world]) as numpy arrays."""
    import numpy as np

    owner = np.empty(window_count(grid, win, shift), dtype=np.int32)
    tokens = np.empty(int(world), dtype=np.int64)
    _check(load_library().h3_sp_assign_windows(_i3(grid), _i3(win), _i3(shift), int(world),
                                               _np_ptr(owner), _np_ptr(tokens)), "h3_sp_assign_windows")
    return owner, tokens


def sp_layer_order(grid, win, shift, window_rank, world: int, rank: int):
    """Original token indices a rank holds in one layer, in its local order (numpy int32)."""
    import numpy as np

    owner = np.ascontiguousarray(window_rank, dtype=np.int32)
    n = int(sp_rank_tokens(grid, win, shift, owner, world)[rank])
    order = np.empty(max(n, 1), dtype=np.int32)
    _check(load_library().h3_sp_layer_order(_i3(grid), _i3(win), _i3(shift), _np_ptr(owner), int(world),
                                            int(rank), _np_ptr(order), n), "h3_sp_layer_order")
    return order[:n]


def sp_rank_tokens(grid, win, shift, window_rank, world: int):
    """Tokens each rank owns under a given window -> rank map (numpy int64 [world])."""
    import numpy as np

    owner = np.ascontiguousarray(window_rank, dtype=np.int32)
    tokens = np.empty(int(world), dtype=np.int64)
    _check(load_library().h3_sp_rank_tokens(_i3(grid), _i3(win), _i3(shift), _np_ptr(owner), int(world),
                                            _np_ptr(tokens)), "h3_sp_rank_tokens")
    return tokens


def sp_exchange_plan(grid, win, shift_from, rank_from, shift_to, rank_to, world: int, rank: int):
    """All-to-all of a layer switch seen by one rank: dict of numpy arrays send_counts,
    send_index, recv_counts, recv_position (see h3_sp_exchange_plan)."""
    import numpy as np

    a = np.ascontiguousarray(rank_from, dtype=np.int32)
    b = np.ascontiguousarray(rank_to, dtype=np.int32)
    n_from = int(sp_rank_tokens(grid, win, shift_from, a, world)[rank])
    n_to = int(sp_rank_tokens(grid, win, shift_to, b, world)[rank])
    plan = dict(send_counts=np.empty(int(world), np.int64), send_index=np.empty(max(n_from, 1), np.int32),
                recv_counts=np.empty(int(world), np.int64), recv_position=np.empty(max(n_to, 1), np.int32))
    _check(load_library().h3_sp_exchange_plan(_i3(grid), _i3(win), _i3(shift_from), _np_ptr(a), _i3(shift_to),
                                              _np_ptr(b), int(world), int(rank),
                                              _np_ptr(plan["send_counts"]), _np_ptr(plan["send_index"]),
                                              _np_ptr(plan["recv_counts"]), _np_ptr(plan["recv_position"])),
           "h3_sp_exchange_plan")
    plan["send_index"] = plan["send_index"][:n_from]
    plan["recv_position"] = plan["recv_position"][:n_to]
    return plan


def get_device_error(device: Optional[torch.device] = None) -> int:
    """Synchronise the current stream; return and clear the device error word (0 = none)."""
    dev = device or torch.device("cuda", torch.cuda.current_device())
    lib = load_library()
    with torch.cuda.device(dev):
        return int(lib.h3_get_device_error(_stream(dev)))


def set_wait_limit_ns(nanoseconds: int) -> int:
    """Limit of the attention kernels' internal waits for later launches (0 = the 2 s default);
    returns the previous limit.  A testing hook for the timeout path: see h3_set_wait_limit_ns."""
    return int(load_library().h3_set_wait_limit_ns(int(nanoseconds)))


def debug_stall_loads(tiles: int) -> int:
    """Make each attention CTA's key/value loader stop after `tiles` tiles (negative = never);
    returns the previous setting.  A testing hook for the timeout path: see h3_debug_stall_loads."""
    return int(load_library().h3_debug_stall_loads(int(tiles)))
