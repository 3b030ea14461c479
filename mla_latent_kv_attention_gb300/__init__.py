"""MLA attention over a paged FP8-e4m3 latent KV cache on one GB300 (sm_103a).

A thin ctypes binding over ``libmla.so`` (C ABI in ``include/mla.h``). The functions
carry the C names and only marshal arguments: torch CUDA tensors become device
pointers, the current torch stream becomes the ``cudaStream_t``. A call that is given a
``stream`` makes it the current one for what it allocates (outputs, a workspace), as
``with torch.cuda.stream(stream)`` does: that memory belongs to it. Every step of the
attention runs in the library's CUDA kernels; there is no other implementation, and
every entry point raises ImportError when the library is missing (the seeded workload
and accounting modules import without it).
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmla.so")

MLA_D = 576
MLA_DV = 512
MLA_ROPE = 64
MLA_MAX_TREE = 64
MLA_MAX_VOCAB = 1 << 19
MLA_MAX_AXES = 4
MLA_OP_DECODE, MLA_OP_VERIFY, MLA_OP_PREFILL, MLA_OP_VERIFY_TREE = 0, 1, 2, 3
(MLA_OK, MLA_ERR_INVALID_ARG, MLA_ERR_UNSUPPORTED, MLA_ERR_WORKSPACE, MLA_ERR_CUDA,
 MLA_ERR_TIMEOUT, MLA_ERR_BOUNDS) = range(7)
STATUS = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_WORKSPACE",
          4: "MLA_ERR_CUDA", 5: "MLA_ERR_TIMEOUT", 6: "MLA_ERR_BOUNDS"}

# Every symbol include/mla.h declares.
EXPORTS = ("mla_workspace_size", "mla_decode", "mla_verify", "mla_prefill", "mla_merge_lse",
           "mla_read_status", "mla_status_string", "mla_last_launch_count",
           "mla_set_profile_events", "mla_decode_static_ws", "mla_cache_append",
           "mla_top_k_renorm_prob", "mla_verify_f32", "mla_prefill_mha",
           "mla_prefill_mha_workspace_size", "mla_test_stall_next_call",
           "mla_read_status_static", "mla_set_trace_buffer", "mla_verify_f32_shard",
           "mla_prefill_mha_bf16", "mla_rope_init", "mla_rope", "mla_cache_append_rope",
           "mla_cache_gather", "mla_verify_tree", "mla_accept_drafts", "mla_rope_axes_init",
           "mla_rope_axes", "mla_cache_append_rope_axes", "mla_cache_append_scaled",
           "mla_cache_gather_scaled", "mla_decode_scaled", "mla_verify_scaled",
           "mla_verify_tree_scaled", "mla_prefill_scaled", "mla_prefill_mha_scaled")


_BLOCKS = (1, 2, 4, 8, 16, 32, 64)
_U8, _I32, _I64, _F32, _BF16 = (torch.uint8, torch.int32, torch.int64, torch.float32,
                                torch.bfloat16)


class MlaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {STATUS.get(status, status)}: "
                         f"{library().mla_status_string(status).decode()}")


class mla_kv_t(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("page_table", ctypes.c_void_p),
                ("page_table_stride", ctypes.c_int64), ("seq_lens", ctypes.c_void_p),
                ("kv_scale", ctypes.c_float)]


class mla_scales_t(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_void_p), ("block", ctypes.c_int32)]


class mla_rope_t(ctypes.Structure):
    """Rotary frequencies as mla_rope_init fills them (see include/mla.h)."""
    _fields_ = [("turns", ctypes.c_uint64 * (MLA_ROPE // 2)), ("amplitude", ctypes.c_float),
                ("interleaved", ctypes.c_int32)]


class mla_rope_axes_t(ctypes.Structure):
    """The position axis of each RoPE pair as mla_rope_axes_init fills it (see include/mla.h)."""
    _fields_ = [("axis", ctypes.c_uint8 * (MLA_ROPE // 2)), ("n_axes", ctypes.c_int32)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmla.so not built at {LIB_PATH}: run "
                          "`python -c 'import __graft_entry__ as g; g.build()'` first")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                            ctypes.c_size_t)
    KV = ctypes.POINTER(mla_kv_t)
    lib.mla_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.mla_workspace_size.restype = sz
    lib.mla_decode.argtypes = [KV, P, i32, i32, f32, P, P, P, sz, P]
    lib.mla_verify.argtypes = [KV, P, i32, i32, i32, f32, P, P, P, sz, P]
    lib.mla_verify_f32.argtypes = [KV, P, i32, i32, i32, f32, P, P, P, sz, P]
    lib.mla_verify_f32.restype = i32
    lib.mla_verify_f32_shard.argtypes = [KV, P, i32, i32, i32, f32, i32, P, P, P, sz, P]
    lib.mla_verify_f32_shard.restype = i32
    lib.mla_prefill_mha_workspace_size.argtypes = [i32, i32, i32]
    lib.mla_prefill_mha_workspace_size.restype = sz
    lib.mla_prefill_mha.argtypes = [KV, i32, P, i32, i32, P, f32, P, P, P, sz, P]
    lib.mla_prefill_mha.restype = i32
    lib.mla_prefill_mha_bf16.argtypes = [KV, i32, P, i32, i32, P, f32, P, P, P, sz, P]
    lib.mla_prefill_mha_bf16.restype = i32
    lib.mla_test_stall_next_call.argtypes = []
    lib.mla_test_stall_next_call.restype = None
    lib.mla_prefill.argtypes = [KV, P, i32, i32, f32, P, P, P, sz, P]
    lib.mla_merge_lse.argtypes = [P, P, i32, i64, P, P, P]
    lib.mla_read_status.argtypes = [P, sz, P]
    lib.mla_status_string.argtypes = [i32]
    lib.mla_status_string.restype = ctypes.c_char_p
    lib.mla_last_launch_count.argtypes = []
    lib.mla_set_profile_events.argtypes = [P, P]
    lib.mla_set_profile_events.restype = None
    lib.mla_decode_static_ws.argtypes = [KV, P, i32, i32, f32, P, P, P]
    lib.mla_decode_static_ws.restype = i32
    lib.mla_read_status_static.argtypes = [P]
    lib.mla_read_status_static.restype = i32
    lib.mla_set_trace_buffer.argtypes = [P, sz]
    lib.mla_set_trace_buffer.restype = None
    lib.mla_cache_append.argtypes = [P, i64, i32, P, P, i64, f32, P, P]
    lib.mla_cache_append.restype = i32
    lib.mla_top_k_renorm_prob.argtypes = [P, P, i32, i32, P, i32, P]
    lib.mla_top_k_renorm_prob.restype = i32
    ROPE = ctypes.POINTER(mla_rope_t)
    f64 = ctypes.c_double
    lib.mla_rope_init.argtypes = [ROPE, f64, f64, i32, f64, f64, f32, i32]
    lib.mla_rope.argtypes = [ROPE, P, i64, i64, P, i64, i32, P, i64, i64, P]
    lib.mla_cache_append_rope.argtypes = [P, i64, i32, P, i64, P, i64, f32, P, f32, ROPE, P, P, P]
    lib.mla_cache_gather.argtypes = [KV, i32, P, P, i64, P, i32, P, P]
    lib.mla_verify_tree.argtypes = [KV, P, i32, i32, i32, f32, P, P, P, P, sz, P]
    lib.mla_accept_drafts.argtypes = [P, P, P, P, P, i32, i32, i32, P, P, P, P]
    AXES = ctypes.POINTER(mla_rope_axes_t)
    lib.mla_rope_axes_init.argtypes = [AXES, ctypes.POINTER(ctypes.c_int32), i32, i32]
    lib.mla_rope_axes.argtypes = [ROPE, AXES, P, i64, i64, P, i64, i32, P, i64, i64, P]
    lib.mla_cache_append_rope_axes.argtypes = [P, i64, i32, P, i64, P, i64, f32, P, f32, ROPE, AXES, P, P, P]
    SCALES = ctypes.POINTER(mla_scales_t)
    lib.mla_cache_append_scaled.argtypes = [KV, SCALES, P, i64, P, i32, i64, P, f32, ROPE, AXES, P, P, P]
    lib.mla_cache_gather_scaled.argtypes = [KV, SCALES, i32, P, P, i64, P, i32, P, P]
    lib.mla_decode_scaled.argtypes = [KV, SCALES, P, i32, i32, f32, P, P, P, sz, P]
    lib.mla_verify_scaled.argtypes = [KV, SCALES, P, i32, i32, i32, f32, i32, P, i32, P, P, sz, P]
    lib.mla_verify_tree_scaled.argtypes = [KV, SCALES, P, i32, i32, i32, f32, P, P, P, P, sz, P]
    lib.mla_prefill_scaled.argtypes = [KV, SCALES, P, i32, i32, f32, P, P, P, sz, P]
    lib.mla_prefill_mha_scaled.argtypes = [KV, SCALES, i32, P, i32, i32, P, f32, i32, P, P, P, sz, P]
    for name in ("mla_rope_init", "mla_rope", "mla_cache_append_rope", "mla_cache_gather",
                 "mla_verify_tree", "mla_accept_drafts", "mla_rope_axes_init", "mla_rope_axes",
                 "mla_cache_append_rope_axes", "mla_cache_append_scaled", "mla_cache_gather_scaled",
                 "mla_decode_scaled", "mla_verify_scaled", "mla_verify_tree_scaled", "mla_prefill_scaled",
                 "mla_prefill_mha_scaled"):
        getattr(lib, name).restype = i32
    for name in ("mla_decode", "mla_verify", "mla_prefill", "mla_merge_lse", "mla_read_status",
                 "mla_last_launch_count"):
        getattr(lib, name).restype = i32
    return lib


_lib: Optional[ctypes.CDLL] = None


def library() -> ctypes.CDLL:
    """The loaded libmla.so (loaded on first use; raises ImportError if not built)."""
    global _lib
    if _lib is None:
        _lib = _load()
    return _lib


@dataclasses.dataclass
class KVCache:
    """Device-resident paged latent cache (see ``mla_kv_t`` in include/mla.h).
    pool uint8 [num_pages, page_size, 576]; page_table int32 [B, stride]; seq_lens int32 [B].
    A cache with a scale for each block of positions (``mla_scales_t``) has ``scales`` float32
    [num_pages, page_size / block], block 1, 2, 4, .. 64, in the place of kv_scale, which is then 1;
    every call that takes a KVCache reads it under them."""

    pool: torch.Tensor
    page_table: torch.Tensor
    seq_lens: torch.Tensor
    kv_scale: float
    scales: Optional[torch.Tensor] = None

    def c_scales(self) -> Optional[mla_scales_t]:
        """The block scales, or None for a cache with one scale (after c_struct's checks)."""
        t = self.scales
        if t is None:
            return None
        pool = self.pool
        if t.dtype is not _F32 or not t.is_contiguous() or t.get_device() != pool.get_device():
            raise ValueError("KVCache.scales must be a contiguous float32 tensor on the pool's device")
        shape, (pages, size, *_) = t.shape, pool.shape
        block = size // shape[1] if len(shape) == 2 and shape[1] > 0 else 0
        if block not in _BLOCKS or shape[0] != pages or block * shape[1] != size:
            raise ValueError("KVCache.scales must be [num_pages, page_size / block] for blocks of 1, 2, 4, .. 64 "
                             f"positions, got {tuple(shape)} for {pages} pages of {size}")
        if float(self.kv_scale) != 1.0:
            raise ValueError("a KVCache with block scales has kv_scale 1 (it is not read)")
        return mla_scales_t(t.data_ptr(), block)

    def c_struct(self) -> mla_kv_t:
        pool, table, lens = self.pool, self.page_table, self.seq_lens
        if not (pool.is_contiguous() and table.is_contiguous() and lens.is_contiguous() and
                pool.get_device() == table.get_device() == lens.get_device() >= 0):
            for name, t in (("pool", pool), ("page_table", table), ("seq_lens", lens)):
                if not t.is_cuda or not t.is_contiguous():
                    raise ValueError(f"KVCache.{name} must be a contiguous CUDA tensor")
            raise ValueError("KVCache tensors must be on one device")
        if pool.dtype is not _U8 or table.dtype is not _I32 or lens.dtype is not _I32:
            raise TypeError("KVCache dtypes: pool uint8, page_table int32, seq_lens int32")
        shape, rows = pool.shape, table.shape
        if (len(shape) != 3 or shape[2] != MLA_D) and (len(shape) < 3 or shape[2:].numel() != MLA_D):
            raise ValueError(f"KVCache.pool must be [num_pages, page_size, {MLA_D}], got {tuple(shape)}")
        if len(rows) != 2 and (len(rows) < 2 or rows[2:].numel() != 1):
            raise ValueError(f"KVCache.page_table must be [B, stride], got {tuple(rows)}")
        return mla_kv_t(pool.data_ptr(), shape[0], shape[1], table.data_ptr(), rows[1],
                        lens.data_ptr(), float(self.kv_scale))

    @staticmethod
    def from_inputs(inp, device="cuda") -> "KVCache":
        return KVCache(inp.pool.to(device), inp.page_table.to(device), inp.seq_lens.to(device),
                       inp.kv_scale)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:  # the current stream's handle (as torch.cuda.current_stream() has it)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise MlaError(fn, status)


def mla_workspace_size(op: int, B: int, H: int, n_q: int, device: Optional[int] = None) -> int:
    if device is None:
        device = torch.cuda.current_device()
    return int(library().mla_workspace_size(op, B, H, n_q, device))


def workspace(op: int, B: int, H: int, n_q: int, device=None) -> torch.Tensor:
    """A zero-filled uint8 device buffer of the size mla_workspace_size() asks for."""
    n = mla_workspace_size(op, B, H, n_q, None if device is None else torch.device(device).index)
    if n == 0:
        raise ValueError("unsupported arguments for mla_workspace_size")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _q_check(q: torch.Tensor, ndim: int) -> None:
    if not q.is_cuda or q.dtype != torch.bfloat16 or not q.is_contiguous() or q.dim() != ndim or \
            q.shape[-1] != MLA_D:
        raise ValueError(f"q must be a contiguous CUDA bfloat16 tensor of rank {ndim} "
                         f"with last dimension {MLA_D}")


def _cache_of(kv: KVCache, q: torch.Tensor, B: int = 1):
    """kv's C structs for a call on q's B sequences, which has to lie on kv's device, the current one
    (the library launches there)."""
    c, scales = kv.c_struct(), kv.c_scales()
    if kv.seq_lens.shape[0] < B or kv.page_table.shape[0] < B:
        raise ValueError(f"kv describes {kv.seq_lens.shape[0]} lengths and {kv.page_table.shape[0]} rows of pages, "
                         f"q has {B} sequences")
    if not kv.pool.get_device() == q.get_device() == torch._C._cuda_getDevice():
        raise ValueError(f"the cache on {kv.pool.device}, q on {q.device}, the current device "
                         f"cuda:{torch._C._cuda_getDevice()}: they have to be one")
    return c, scales


def mla_decode(kv: KVCache, q: torch.Tensor, sm_scale: float, out=None, lse=None, ws=None,
               stream=None):
    """q [B, H, 576] bf16 -> (out [B, H, 512] bf16, lse [B, H] fp32)."""
    if stream is not None and (out is None or lse is None or ws is None):
        with _current(stream):
            return mla_decode(kv, q, sm_scale, out, lse, ws)
    _q_check(q, 3)
    B, H = q.shape[0], q.shape[1]
    c, scales = _cache_of(kv, q, B)
    ws = workspace(MLA_OP_DECODE, B, H, 1, q.device) if ws is None else ws
    out = torch.empty(B, H, MLA_DV, dtype=torch.bfloat16, device=q.device) if out is None else out
    lse = torch.empty(B, H, dtype=torch.float32, device=q.device) if lse is None else lse
    args = (q.data_ptr(), B, H, sm_scale, out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(), _stream(stream))
    if scales is None:
        _check("mla_decode", library().mla_decode(c, *args))
    else:
        _check("mla_decode_scaled", library().mla_decode_scaled(c, scales, *args))
    return out, lse


def mla_verify(kv: KVCache, q: torch.Tensor, sm_scale: float, out=None, lse=None, ws=None,
               stream=None):
    """q [B, n_q, H, 576] bf16 -> (out [B, n_q, H, 512] bf16, lse [B, n_q, H] fp32)."""
    if stream is not None and (out is None or lse is None or ws is None):
        with _current(stream):
            return mla_verify(kv, q, sm_scale, out, lse, ws)
    _q_check(q, 4)
    B, n_q, H = q.shape[0], q.shape[1], q.shape[2]
    c, scales = _cache_of(kv, q, B)
    ws = workspace(MLA_OP_VERIFY, B, H, n_q, q.device) if ws is None else ws
    out = torch.empty(B, n_q, H, MLA_DV, dtype=torch.bfloat16, device=q.device) if out is None else out
    lse = torch.empty(B, n_q, H, dtype=torch.float32, device=q.device) if lse is None else lse
    if scales is None:
        _check("mla_verify", library().mla_verify(ctypes.byref(c), q.data_ptr(), B, n_q, H, sm_scale,
                                             out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(),
                                             _stream(stream)))
    else:
        _check("mla_verify_scaled", library().mla_verify_scaled(
            c, scales, q.data_ptr(), B, n_q, H, sm_scale, 0, out.data_ptr(), 0, _ptr(lse), ws.data_ptr(),
            ws.numel(), _stream(stream)))
    return out, lse


def mla_prefill_mha(kv: KVCache, q: torch.Tensor, w_ukv: torch.Tensor, sm_scale: float,
                    L: Optional[int] = None, out=None, lse=None, ws=None, stream=None,
                    bf16: bool = False):
    """MHA-form causal prefill of sequence 0: q [T, H, 192] bf16, w_ukv [512, H, 256] bf16
    -> (out [T, H, 128] bf16, lse [T, H] fp32). L (cached positions incl. the T new ones)
    defaults to kv.seq_lens[0]. bf16=True calls mla_prefill_mha_bf16 (every tensor-core
    operand in bf16: faster, looser)."""
    if stream is not None and (L is None or out is None or lse is None or ws is None):
        with _current(stream):
            return mla_prefill_mha(kv, q, w_ukv, sm_scale, L, out, lse, ws, bf16=bf16)
    if q.dtype != torch.bfloat16 or q.dim() != 3 or q.shape[2] != 192 or not q.is_contiguous():
        raise ValueError("q must be a contiguous bfloat16 tensor [T, H, 192]")
    T, H = q.shape[0], q.shape[1]
    if w_ukv.dtype != torch.bfloat16 or tuple(w_ukv.shape) != (512, H, 256) or not w_ukv.is_contiguous():
        raise ValueError("w_ukv must be a contiguous bfloat16 tensor [512, H, 256]")
    if L is None:
        L = int(kv.seq_lens[0].item())
    out = torch.empty(T, H, 128, dtype=torch.bfloat16, device=q.device) if out is None else out
    lse = torch.empty(T, H, dtype=torch.float32, device=q.device) if lse is None else lse
    if ws is None:
        n = int(library().mla_prefill_mha_workspace_size(L, H, q.device.index or 0))
        if n == 0:
            raise ValueError("no workspace size for these arguments")
        ws = torch.zeros(n, dtype=torch.uint8, device=q.device)
    c, scales = _cache_of(kv, q)
    name = "mla_prefill_mha_bf16" if bf16 else "mla_prefill_mha"
    tail = (out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(), _stream(stream))
    if scales is None:
        _check(name, getattr(library(), name)(c, L, q.data_ptr(), T, H, w_ukv.data_ptr(), sm_scale, *tail))
    else:
        _check("mla_prefill_mha_scaled", library().mla_prefill_mha_scaled(
            c, scales, L, q.data_ptr(), T, H, w_ukv.data_ptr(), sm_scale, int(bf16), *tail))
    return out, lse


def mla_verify_f32(kv: KVCache, q: torch.Tensor, sm_scale: float, out=None, lse=None, ws=None,
                   stream=None, visible_shift: int = 0):
    """As mla_verify with a float32 output [B, n_q, H, 512], for results merged later.
    visible_shift > 0 moves every new position's causal limit that many keys later
    (mla_verify_f32_shard; n_q - 1 makes every key of the view visible to all of them)."""
    if stream is not None and (out is None or lse is None or ws is None):
        with _current(stream):
            return mla_verify_f32(kv, q, sm_scale, out, lse, ws, visible_shift=visible_shift)
    _q_check(q, 4)
    B, n_q, H = q.shape[0], q.shape[1], q.shape[2]
    out = torch.empty(B, n_q, H, MLA_DV, dtype=torch.float32, device=q.device) if out is None else out
    if out.dtype != torch.float32 or not out.is_contiguous() or out.shape != (B, n_q, H, MLA_DV):
        raise ValueError("out must be a contiguous float32 tensor [B, n_q, H, 512]")
    lse = torch.empty(B, n_q, H, dtype=torch.float32, device=q.device) if lse is None else lse
    ws = workspace(MLA_OP_VERIFY, B, H, n_q, q.device) if ws is None else ws
    c, scales = _cache_of(kv, q, B)
    if scales is not None:
        _check("mla_verify_scaled", library().mla_verify_scaled(
            c, scales, q.data_ptr(), B, n_q, H, sm_scale, int(visible_shift), out.data_ptr(), 1, _ptr(lse),
            ws.data_ptr(), ws.numel(), _stream(stream)))
    elif visible_shift == 0:
        _check("mla_verify_f32", library().mla_verify_f32(
            ctypes.byref(c), q.data_ptr(), B, n_q, H, sm_scale, out.data_ptr(), _ptr(lse),
            ws.data_ptr(), ws.numel(), _stream(stream)))
    else:
        _check("mla_verify_f32_shard", library().mla_verify_f32_shard(
            ctypes.byref(c), q.data_ptr(), B, n_q, H, sm_scale, int(visible_shift),
            out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(), _stream(stream)))
    return out, lse


def mla_prefill(kv: KVCache, q: torch.Tensor, sm_scale: float, out=None, lse=None, ws=None,
                stream=None):
    """q [T, H, 576] bf16 of one sequence -> (out [T, H, 512] bf16, lse [T, H] fp32)."""
    if stream is not None and (out is None or lse is None or ws is None):
        with _current(stream):
            return mla_prefill(kv, q, sm_scale, out, lse, ws)
    _q_check(q, 3)
    T, H = q.shape[0], q.shape[1]
    c, scales = _cache_of(kv, q)
    ws = workspace(MLA_OP_PREFILL, 1, H, T, q.device) if ws is None else ws
    out = torch.empty(T, H, MLA_DV, dtype=torch.bfloat16, device=q.device) if out is None else out
    lse = torch.empty(T, H, dtype=torch.float32, device=q.device) if lse is None else lse
    args = (q.data_ptr(), T, H, sm_scale, out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(), _stream(stream))
    if scales is None:
        _check("mla_prefill", library().mla_prefill(c, *args))
    else:
        _check("mla_prefill_scaled", library().mla_prefill_scaled(c, scales, *args))
    return out, lse


def mla_merge_lse(part_out: torch.Tensor, part_lse: torch.Tensor, out=None, lse=None,
                  stream=None):
    """part_out [S, R, 512] fp32, part_lse [S, R] fp32 -> (out [R, 512] bf16, lse [R] fp32)."""
    if stream is not None and (out is None or lse is None):
        with _current(stream):
            return mla_merge_lse(part_out, part_lse, out, lse)
    if part_out.dtype != torch.float32 or part_lse.dtype != torch.float32 or \
            not part_out.is_contiguous() or not part_lse.is_contiguous():
        raise ValueError("partials must be contiguous float32 CUDA tensors")
    S, R = part_lse.shape
    out = torch.empty(R, MLA_DV, dtype=torch.bfloat16, device=part_out.device) if out is None else out
    lse = torch.empty(R, dtype=torch.float32, device=part_out.device) if lse is None else lse
    _check("mla_merge_lse", library().mla_merge_lse(part_out.data_ptr(), part_lse.data_ptr(), S, R,
                                               out.data_ptr(), _ptr(lse), _stream(stream)))
    return out, lse


def mla_cache_append(pool: torch.Tensor, x: torch.Tensor, slots: torch.Tensor, kv_scale: float,
                     status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write bf16 rows x [n, 576] into the uint8 pool [num_pages, page_size, 576] as e4m3
    codes of x / kv_scale at flat rows `slots` (int64 [n]; negative = skip). `status`, an
    int32 CUDA tensor of one element, receives MLA_ERR_BOUNDS for a slot past the pool."""
    if pool.dtype != torch.uint8 or pool.dim() != 3 or pool.shape[2] != MLA_D or not pool.is_contiguous():
        raise ValueError("pool must be a contiguous uint8 tensor [num_pages, page_size, 576]")
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != MLA_D or not x.is_contiguous():
        raise ValueError("x must be a contiguous bfloat16 tensor [n, 576]")
    if slots.dtype != torch.int64 or slots.dim() != 1 or slots.shape[0] != x.shape[0]:
        raise ValueError("slots must be an int64 tensor [n]")
    _check("mla_cache_append", library().mla_cache_append(
        pool.data_ptr(), pool.shape[0], pool.shape[1], x.data_ptr(), slots.data_ptr(),
        x.shape[0], float(kv_scale), None if status is None else status.data_ptr(),
        _stream(stream)))


def mla_top_k_renorm_prob(probs: torch.Tensor, top_k, out: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """probs float32 [B, V] -> top-k renormalised copy; top_k an int (all rows) or an int32
    CUDA tensor [B]."""
    if stream is not None and out is None:
        with _current(stream):
            return mla_top_k_renorm_prob(probs, top_k)
    if probs.dtype != torch.float32 or probs.dim() != 2 or not probs.is_contiguous():
        raise ValueError("probs must be a contiguous float32 tensor [B, V]")
    B, V = probs.shape
    out = torch.empty_like(probs) if out is None else out
    if isinstance(top_k, torch.Tensor):
        if top_k.dtype != torch.int32 or top_k.shape != (B,):
            raise ValueError("top_k must be an int32 tensor [B]")
        kp, k = top_k.data_ptr(), 0
    else:
        kp, k = None, int(top_k)
    _check("mla_top_k_renorm_prob", library().mla_top_k_renorm_prob(
        probs.data_ptr(), out.data_ptr(), B, V, kp, k, _stream(stream)))
    return out


def _current(stream):
    """Makes `stream` (a torch stream or a raw handle) and its device the current ones, so that
    what a call allocates belongs to the stream that the call runs on. The handles 0 and 1
    (cudaStreamLegacy) are the default stream's; torch would take a new stream from its pool for 0."""
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _on(dev: torch.device) -> int:
    """The raw current stream for a call on tensors of device `dev` (which has to be the current
    one: the library launches on the current device)."""
    index = torch._C._cuda_getDevice()
    if dev.index != index:
        raise ValueError(f"tensors on {dev}, but cuda:{index} is the current device "
                         "(use torch.cuda.device)")
    return torch._C._cuda_getCurrentRawStream(index)


def _dense(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, dev: torch.device) -> int:
    """Pointer of a contiguous tensor of the given type, shape and device."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == dev:
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _status_ptr(status: Optional[torch.Tensor], dev: torch.device) -> Optional[int]:
    return None if status is None else _dense(status, "status", _I32, (1,), dev)


def mla_rope_init(base: float = 10000.0, factor: float = 1.0, original_positions: int = 0,
                  beta_fast: float = 32.0, beta_slow: float = 1.0, amplitude: float = 1.0,
                  interleaved: bool = True) -> mla_rope_t:
    """Rotary frequencies f_i = base^(-2i/64) of the 64 RoPE dims, for a context stretched
    `factor` times: linearly (original_positions = 0) or by YaRN. Kept by the caller and
    handed to mla_rope and mla_cache_append_rope."""
    rope = mla_rope_t()
    _check("mla_rope_init", library().mla_rope_init(rope, base, factor, original_positions, beta_fast,
                                               beta_slow, amplitude, int(interleaved)))
    return rope


def mla_rope_axes_init(sections, interleaved: bool = False) -> mla_rope_axes_t:
    """Positions with several axes (time, height, width): `sections` gives the number of RoPE pairs
    (32 in all) that each axis turns, one section after the other or, interleaved, the axes taking
    pairs in turn while they have any left. Kept by the caller and handed to mla_rope and the cache
    writes with positions int64 [len(sections), n]."""
    axes = mla_rope_axes_t()
    sections = [max(-1, min(int(k), MLA_ROPE)) for k in sections]  # (the C entry's int32 would wrap)
    _check("mla_rope_axes_init", library().mla_rope_axes_init(
        axes, (ctypes.c_int32 * len(sections))(*sections), len(sections), int(interleaved)))
    return axes


def _positions_ptr(positions: Optional[torch.Tensor], axes: Optional[mla_rope_axes_t], n: int,
                   dev: torch.device) -> Optional[int]:
    """Pointer of positions int64 [n], or [axes, n]."""
    if positions is None:
        if axes is not None:
            raise ValueError("axes need positions")
        return None
    return _dense(positions, "positions", _I64, (n,) if axes is None else (axes.n_axes, n), dev)


def _rope_part(t: torch.Tensor, name: str):
    """Shape and strides of a view of the RoPE dims."""
    if t.dtype is _BF16 and t.dim() == 3 and t.is_cuda:
        n, H, width = t.shape
        st, sh, sd = t.stride()
        if width == MLA_ROPE and sd == 1:
            return n, H, st if n > 1 else 0, sh if H > 1 else 0  # (one token, one head: no stride)
    raise ValueError(f"{name} must be a bfloat16 CUDA tensor [n, H, 64] (any token and head "
                     "strides, the 64 RoPE dims contiguous)")


def mla_rope(rope: mla_rope_t, x: torch.Tensor, positions: torch.Tensor, out=None,
             stream=None, axes: Optional[mla_rope_axes_t] = None) -> torch.Tensor:
    """Rotate x [n, H, 64] bf16 (a view of the RoPE dims, e.g. q[..., 512:] or q_mha[..., 128:])
    to positions int64 [n], or [axes.n_axes, n] where `axes` says which axis each pair turns by.
    `out` may be another such view, or x itself (in place)."""
    if stream is not None:
        with _current(stream):
            return mla_rope(rope, x, positions, out, axes=axes)
    n, H, xt, xh = _rope_part(x, "x")
    dev = x.device
    if out is None:
        out = torch.empty((n, H, MLA_ROPE), dtype=_BF16, device=dev)
    m, G, ot, oh = _rope_part(out, "out")
    if m != n or G != H or out.device != dev or (n > 1 and ot == 0) or (H > 1 and oh == 0):
        raise ValueError("out must have x's shape and device, and a place of its own for every element")
    if axes is None:
        _check("mla_rope", library().mla_rope(
            rope, x.data_ptr(), xt, xh, _dense(positions, "positions", _I64, (n,), dev), n, H,
            out.data_ptr(), ot, oh, _on(dev)))
    else:
        _check("mla_rope_axes", library().mla_rope_axes(
            rope, axes, x.data_ptr(), xt, xh, _positions_ptr(positions, axes, n, dev), n, H,
            out.data_ptr(), ot, oh, _on(dev)))
    return out


def mla_cache_append_rope(pool: torch.Tensor, x: torch.Tensor, slots: torch.Tensor, kv_scale: float,
                          rope: Optional[mla_rope_t] = None, positions: Optional[torch.Tensor] = None,
                          norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          status: Optional[torch.Tensor] = None, stream=None,
                          axes: Optional[mla_rope_axes_t] = None) -> None:
    """mla_cache_append for rows x [n, 576] bf16 as the latent projection leaves them: the
    latent is normalised by its root mean square and weighted with norm_weight [512] bf16
    (None: as it is), the 64 RoPE dims are turned to positions int64 [n] (with `axes`,
    [axes.n_axes, n]; rope None: as they are), and both are quantised in one pass. x may be a
    slice of a wider projection's rows."""
    if stream is not None:
        with _current(stream):
            return mla_cache_append_rope(pool, x, slots, kv_scale, rope, positions, norm_weight, eps, status,
                                         axes=axes)
    if pool.dtype is not _U8 or pool.dim() != 3 or not pool.is_contiguous() or not pool.is_cuda or \
            pool.shape[2] != MLA_D:
        raise ValueError("pool must be a contiguous uint8 CUDA tensor [num_pages, page_size, 576]")
    pages, size, _ = pool.shape
    dev = pool.device
    n, stride = _latent_rows(x, dev)
    if (rope is None) != (positions is None):
        raise ValueError("give rope and positions together, or neither")
    args = (pool.data_ptr(), pages, size, x.data_ptr(), stride, _dense(slots, "slots", _I64, (n,), dev), n, kv_scale,
            None if norm_weight is None else _dense(norm_weight, "norm_weight", _BF16, (MLA_DV,), dev), eps, rope)
    at, word = _positions_ptr(positions, axes, n, dev), _status_ptr(status, dev)
    if axes is None:
        _check("mla_cache_append_rope", library().mla_cache_append_rope(*args, at, word, _on(dev)))
    else:
        _check("mla_cache_append_rope_axes", library().mla_cache_append_rope_axes(*args, axes, at, word, _on(dev)))


def _latent_rows(x: torch.Tensor, dev: torch.device):
    """Number and stride of rows x [n, 576] that a cache write takes."""
    if x.dtype is not _BF16 or x.dim() != 2 or x.shape[1] != MLA_D or x.stride(1) != 1 or \
            x.device != dev:
        raise ValueError("x must be a bfloat16 tensor [n, 576] on the pool's device, its rows contiguous")
    n = x.shape[0]
    return n, x.stride(0) if n > 1 else MLA_D


def mla_cache_append_scaled(kv: KVCache, x: torch.Tensor, cu_rows: torch.Tensor,
                            rope: Optional[mla_rope_t] = None, positions: Optional[torch.Tensor] = None,
                            axes: Optional[mla_rope_axes_t] = None, norm_weight: Optional[torch.Tensor] = None,
                            eps: float = 1e-6, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write new rows x [n, 576] bf16, as the latent projection leaves them, into a cache with block
    scales, choosing the scales: rows cu_rows[b] .. cu_rows[b + 1] - 1 (int64 [B + 1]) are the last
    of sequence b's kv.seq_lens[b] positions. Norm, rotation and arguments otherwise as
    mla_cache_append_rope; kv.pool and kv.scales are written. A block's scale grows to the power of
    two that its new rows need, its earlier rows' codes with it."""
    if stream is not None:
        with _current(stream):
            return mla_cache_append_scaled(kv, x, cu_rows, rope, positions, axes, norm_weight, eps, status)
    c = kv.c_struct()
    scales = kv.c_scales()
    if scales is None:
        raise ValueError("kv has no block scales (KVCache.scales)")
    dev = kv.pool.device
    n, stride = _latent_rows(x, dev)
    B = cu_rows.shape[0] - 1 if cu_rows.dim() == 1 else -1
    if B < 0 or B > kv.seq_lens.shape[0] or B > kv.page_table.shape[0]:
        raise ValueError("cu_rows must have an entry more than there are sequences")
    if (rope is None) != (positions is None):
        raise ValueError("give rope and positions together, or neither")
    _check("mla_cache_append_scaled", library().mla_cache_append_scaled(
        c, scales, x.data_ptr(), stride, _dense(cu_rows, "cu_rows", _I64, (B + 1,), dev), B, n,
        None if norm_weight is None else _dense(norm_weight, "norm_weight", _BF16, (MLA_DV,), dev), eps, rope, axes,
        _positions_ptr(positions, axes, n, dev), _status_ptr(status, dev), _on(dev)))


def mla_cache_gather(kv: KVCache, cu_rows: torch.Tensor, n: int, starts: Optional[torch.Tensor] = None,
                     out=None, dtype: torch.dtype = torch.bfloat16,
                     status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Cached rows read back and dequantised: rows cu_rows[b] .. cu_rows[b + 1] - 1 of out
    [n, 576] (bf16 or float32) are positions starts[b], starts[b] + 1, ... of sequence b.
    cu_rows int64 [B + 1], starts int32 [B] (None: 0); rows outside them stay as they were. A cache
    with block scales is read under them."""
    if stream is not None:
        with _current(stream):
            return mla_cache_gather(kv, cu_rows, n, starts, out, dtype, status)
    c = kv.c_struct()
    dev = kv.pool.device
    B = cu_rows.shape[0] - 1
    if B < 0 or B > kv.seq_lens.shape[0] or B > kv.page_table.shape[0]:
        raise ValueError("cu_rows must have an entry more than there are sequences")
    f32 = (dtype if out is None else out.dtype) is _F32
    if not f32 and out is None and dtype is not _BF16:
        raise ValueError("dtype must be bfloat16 or float32")
    cu_ptr = _dense(cu_rows, "cu_rows", _I64, (B + 1,), dev)
    starts_ptr = None if starts is None else _dense(starts, "starts", _I32, (B,), dev)
    scales, word, current = kv.c_scales(), _status_ptr(status, dev), _on(dev)
    if out is None:
        out = torch.empty((n, MLA_D), dtype=dtype, device=dev)
    else:
        _dense(out, "out", _F32 if f32 else _BF16, (n, MLA_D), dev)
    args = (B, starts_ptr, cu_ptr, n, out.data_ptr(), f32, word, current)
    if scales is None:
        _check("mla_cache_gather", library().mla_cache_gather(c, *args))
    else:
        _check("mla_cache_gather_scaled", library().mla_cache_gather_scaled(c, scales, *args))
    return out


def mla_verify_tree(kv: KVCache, q: torch.Tensor, tree_mask: torch.Tensor, sm_scale: float, out=None,
                    lse=None, ws=None, stream=None):
    """q [B, n, H, 576] bf16 of a tree's n <= 64 nodes -> (out [B, n, H, 512] bf16, lse [B, n, H]
    fp32). Every node sees the prefix and the nodes whose bit its tree_mask (int64 [B, n]) sets."""
    if stream is not None:
        with _current(stream):
            return mla_verify_tree(kv, q, tree_mask, sm_scale, out, lse, ws)
    _q_check(q, 4)
    B, n, H, _ = q.shape
    dev = q.device
    c, scales = kv.c_struct(), kv.c_scales()
    if kv.seq_lens.shape[0] < B or kv.page_table.shape[0] < B or kv.pool.device != dev:
        raise ValueError("kv must describe q's sequences, on q's device")
    mask, current = _dense(tree_mask, "tree_mask", _I64, (B, n), dev), _on(dev)
    if ws is None:
        ws = workspace(MLA_OP_VERIFY_TREE, B, H, n, dev)
    elif ws.dtype is not _U8 or not ws.is_contiguous() or ws.device != dev:
        raise ValueError("ws must be a contiguous uint8 tensor on q's device")
    if out is None:
        out = torch.empty((B, n, H, MLA_DV), dtype=_BF16, device=dev)
    else:
        _dense(out, "out", _BF16, (B, n, H, MLA_DV), dev)
    if lse is None:
        lse = torch.empty((B, n, H), dtype=_F32, device=dev)
    else:
        _dense(lse, "lse", _F32, (B, n, H), dev)
    args = (q.data_ptr(), B, n, H, sm_scale, mask, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), current)
    if scales is None:
        _check("mla_verify_tree", library().mla_verify_tree(c, *args))
    else:
        _check("mla_verify_tree_scaled", library().mla_verify_tree_scaled(c, scales, *args))
    return out, lse


def mla_accept_drafts(target_probs: torch.Tensor, tokens: torch.Tensor, uniforms: torch.Tensor,
                      parents: Optional[torch.Tensor] = None,
                      draft_probs: Optional[torch.Tensor] = None, stream=None):
    """Accept drafted tokens against target_probs [B, n, V] float32 (row j: the token after node
    j) and draw the token after them. tokens int32 [B, n] (node 0 is the last token emitted),
    uniforms float32 [B, n + 1] in [0, 1), parents int32 [B, n] (None: a chain), draft_probs
    float32 [B, n - 1, V] (chains: what tokens[:, 1:] were drawn from). Returns int32 tensors
    (out_tokens [B, n], path [B, n], num_accepted [B]); unused places hold -1."""
    if stream is not None:
        with _current(stream):
            return mla_accept_drafts(target_probs, tokens, uniforms, parents, draft_probs)
    if target_probs.dim() != 3 or not target_probs.is_cuda:
        raise ValueError("target_probs must be a CUDA tensor [B, n, V]")
    B, n, V = target_probs.shape
    dev = target_probs.device
    _dense(tokens, "tokens", _I32, (B, n), dev)
    out_tokens = torch.empty_like(tokens)
    path = torch.empty_like(tokens)
    num_accepted = torch.empty((B,), dtype=_I32, device=dev)
    _check("mla_accept_drafts", library().mla_accept_drafts(
        _dense(target_probs, "target_probs", _F32, (B, n, V), dev), tokens.data_ptr(),
        None if parents is None else _dense(parents, "parents", _I32, (B, n), dev),
        None if draft_probs is None else _dense(draft_probs, "draft_probs", _F32, (B, n - 1, V), dev),
        _dense(uniforms, "uniforms", _F32, (B, n + 1), dev), B, n, V, out_tokens.data_ptr(),
        path.data_ptr(), num_accepted.data_ptr(), _on(dev)))
    return out_tokens, path, num_accepted


def mla_read_status(ws: torch.Tensor, stream=None) -> int:
    return int(library().mla_read_status(ws.data_ptr(), ws.numel(), _stream(stream)))


def mla_last_launch_count() -> int:
    return int(library().mla_last_launch_count())


def mla_set_profile_events(start=None, stop=None) -> None:
    """Record torch.cuda.Event `start`/`stop` around the main attention kernel of the
    following calls on this thread (None, None switches it off)."""
    if (start is None) != (stop is None):
        raise ValueError("give both events or neither")
    library().mla_set_profile_events(None if start is None else start.cuda_event,
                                     None if stop is None else stop.cuda_event)
