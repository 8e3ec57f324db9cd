"""ctypes binding of the C-ABI library (``include/pa.h``).

Argument marshalling only: every function checks tensor devices, dtypes,
shapes and contiguity, then passes raw pointers, sizes and the current CUDA
stream to the library, whose kernels do all the work.  Importing this module
without the built library raises ImportError; there is no fallback path.

Names follow the C ABI: ``pa_decode``, ``pa_decode_workspace_size``,
``pa_reshape_and_cache``, ``pa_copy_blocks`` and the ``BlockManager`` class
over ``pa_bm_*``.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

from . import build as _build

PA_OK = 0
PA_ERR_INVALID_ARG = -1
PA_ERR_UNSUPPORTED = -2
PA_ERR_CUDA = -3
PA_ERR_BAD_INDEX = -4
PA_ERR_NO_BLOCKS = -5
PA_ERR_REFCOUNT = -6
PA_ERR_WORKSPACE = -7

PA_F32, PA_BF16 = 0, 1
PA_PHASE_ALL, PA_PHASE_PARTITIONS, PA_PHASE_REDUCE = 0, 1, 2

STATUS_BAD_BLOCK_ID = 1
STATUS_BAD_CONTEXT_LEN = 2
STATUS_BAD_SLOT = 4
STATUS_BAD_PAIR = 8
STATUS_WAIT_TIMEOUT = 16
STATUS_SHORT_LIST = 32
STATUS_BAD_TREE = 64


class PAError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class _DecodeArgs(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int),
        ("max_blocks_per_seq", ctypes.c_int),
        ("num_blocks", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("partition_size", ctypes.c_int),
        ("max_context_len", ctypes.c_int),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("dev_status", ctypes.c_void_p),
        ("stream", ctypes.c_void_p),
        ("phase", ctypes.c_int),
        ("k_new", ctypes.c_void_p),
        ("v_new", ctypes.c_void_p),
        ("slot_mapping", ctypes.c_void_p),
        ("simt", ctypes.c_int),
        ("skip_counter_reset", ctypes.c_int),
        ("max_query_len", ctypes.c_int),
    ]


def library_path() -> str:
    return _build.LIB_PATH


def _declare(lib: ctypes.CDLL) -> ctypes.CDLL:
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.pa_decode.restype = i32
    lib.pa_decode.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, ctypes.POINTER(_DecodeArgs)]
    lib.pa_decode_noalloc.restype = i32
    lib.pa_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32,
                                      ctypes.POINTER(_DecodeArgs)]
    lib.pa_decode_workspace_size.restype = sz
    lib.pa_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.pa_reshape_and_cache.restype = i32
    lib.pa_reshape_and_cache.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp]
    lib.pa_copy_blocks.restype = i32
    lib.pa_copy_blocks.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp]
    lib.pa_swap_blocks.restype = i32
    lib.pa_swap_blocks.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp]
    lib.pa_bm_move_seq.restype = i32
    lib.pa_bm_move_seq.argtypes = [vp, vp, i32, vp, i32, ctypes.POINTER(i32)]
    lib.pa_selftest_wait_timeout.restype = i32
    lib.pa_selftest_wait_timeout.argtypes = [vp, i32, vp]
    lib.pa_bm_create.restype = vp
    lib.pa_bm_create.argtypes = [i32, i32]
    lib.pa_bm_destroy.restype = None
    lib.pa_bm_destroy.argtypes = [vp]
    lib.pa_bm_add_seq.restype = i32
    lib.pa_bm_add_seq.argtypes = [vp, i32, i32]
    lib.pa_bm_fork.restype = i32
    lib.pa_bm_fork.argtypes = [vp, i32, i32]
    lib.pa_bm_append_slot.restype = i32
    lib.pa_bm_append_slot.argtypes = [vp, i32, ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_int32),
                                      ctypes.POINTER(ctypes.c_int32)]
    lib.pa_bm_free_seq.restype = i32
    lib.pa_bm_free_seq.argtypes = [vp, i32]
    lib.pa_bm_block_table.restype = i32
    lib.pa_bm_block_table.argtypes = [vp, i32, vp, i32]
    lib.pa_bm_num_tokens.restype = i32
    lib.pa_bm_num_tokens.argtypes = [vp, i32]
    lib.pa_bm_num_free.restype = i32
    lib.pa_bm_num_free.argtypes = [vp]
    lib.pa_bm_refcount.restype = i32
    lib.pa_bm_refcount.argtypes = [vp, i32]
    lib.pa_bm_append_slots.restype = i32
    lib.pa_bm_append_slots.argtypes = [vp, vp, i32, vp, vp, ctypes.POINTER(i32), ctypes.POINTER(i32)]
    lib.pa_bm_add_seq_cached.restype = i32
    lib.pa_bm_add_seq_cached.argtypes = [vp, i32, vp, i32, ctypes.c_uint64, ctypes.POINTER(i32)]
    lib.pa_bm_register_blocks.restype = i32
    lib.pa_bm_register_blocks.argtypes = [vp, i32, vp, i32, ctypes.c_uint64]
    lib.pa_bm_num_cached.restype = i32
    lib.pa_bm_num_cached.argtypes = [vp]
    lib.pa_bm_build_tables.restype = i32
    lib.pa_bm_build_tables.argtypes = [vp, vp, i32, vp, i32, vp]
    lib.pa_decode_window.restype = i32
    lib.pa_decode_window.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, i32, i32,
                                     ctypes.POINTER(_DecodeArgs)]
    lib.pa_decode_window_workspace_size.restype = sz
    lib.pa_decode_window_workspace_size.argtypes = [i32] * 9
    lib.pa_decode_q4.restype = i32
    lib.pa_decode_q4.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, i32,
                                 ctypes.POINTER(_DecodeArgs)]
    lib.pa_decode_q4_workspace_size.restype = sz
    lib.pa_decode_q4_workspace_size.argtypes = [i32] * 8
    lib.pa_bm_flat_blocks.restype = i32
    lib.pa_bm_flat_blocks.argtypes = [vp, vp, i32, vp, i32, vp]
    lib.pa_build_tables.restype = i32
    lib.pa_build_tables.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp]
    lib.pa_q4_page_bytes.restype = sz
    lib.pa_q4_page_bytes.argtypes = [i32, i32, i32]
    lib.pa_reshape_and_cache_q4.restype = i32
    lib.pa_reshape_and_cache_q4.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp]
    lib.pa_gather_q4.restype = i32
    lib.pa_gather_q4.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp]
    lib.pa_decode_tree.restype = i32
    lib.pa_decode_tree.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, i32, i32,
                                   ctypes.POINTER(_DecodeArgs)]
    lib.pa_decode_cross.restype = i32
    lib.pa_decode_cross.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, i32,
                                    ctypes.POINTER(_DecodeArgs)]
    lib.pa_decode_tree_workspace_size.restype = sz
    lib.pa_decode_tree_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.pa_build_tree.restype = i32
    lib.pa_build_tree.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, vp, vp]
    lib.pa_accept_tree.restype = i32
    lib.pa_accept_tree.argtypes = [vp] * 11 + [i32] * 6 + [vp, vp]
    lib.pa_move_rows.restype = i32
    lib.pa_move_rows.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp]
    lib.pa_bm_trim_seq.restype = i32
    lib.pa_bm_trim_seq.argtypes = [vp, i32, i32]
    lib.pa_last_error_string.restype = ctypes.c_char_p
    lib.pa_last_error_string.argtypes = []
    lib.pa_version.restype = i32
    lib.pa_version.argtypes = []
    return lib


def load_library() -> ctypes.CDLL:
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run `python -m paged_kv_cache_237_gb300.build` "
                          "or __graft_entry__.build() first")
    return _declare(ctypes.CDLL(path))


_lib = load_library()


def declared_functions(header: str | None = None) -> list[str]:
    """Names of the functions include/pa.h declares (used by the ABI tests)."""
    header = header or os.path.join(_build.INCLUDE, "pa.h")
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(pa_[a-z0-9_]+)\s*\(", text)))


def _raise(rc: int):
    if rc != PA_OK:
        raise PAError(rc, _lib.pa_last_error_string().decode())


def _stream_ptr(stream, device) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: torch.Tensor | None):
    return t.data_ptr() if t is not None else None


_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _call(dev: torch.device, fn, *args) -> None:
    """Calls a library function with dev as the current device."""
    if _current_device() == dev.index:
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc:
        _raise(rc)


def _check_cuda(t: torch.Tensor, name: str, dtypes, dev=None):
    if t.__class__ is torch.Tensor and t.dtype in dtypes and t.is_contiguous() and \
            (t.device == dev if dev is not None else t.is_cuda):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    if dev is not None and t.get_device() != dev.index:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_int32(dev: torch.device, **tensors) -> None:
    """``_check_cuda`` of several int32 tensors on one device."""
    at, i32 = dev.index, torch.int32
    for name, t in tensors.items():
        if not (t.__class__ is torch.Tensor and t.dtype is i32 and t.get_device() == at and t.is_contiguous()):
            _check_cuda(t, name, (i32,), dev)


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return PA_F32
    if dt == torch.bfloat16:
        return PA_BF16
    raise TypeError(f"unsupported dtype {dt}")


class DeviceStatus:
    """A device int32 word that kernels OR PA_STATUS_* bits into."""

    def __init__(self, device="cuda"):
        self.tensor = torch.zeros(1, dtype=torch.int32, device=device)

    def ptr(self) -> int:
        return self.tensor.data_ptr()

    def read(self, clear: bool = True) -> int:
        v = int(self.tensor.item())
        if clear:
            self.tensor.zero_()
        return v


def pa_decode_workspace_size(num_seqs: int, num_q_heads: int, head_dim: int, max_context_len: int,
                             partition_size: int = 0) -> int:
    return int(_lib.pa_decode_workspace_size(num_seqs, num_q_heads, head_dim, max_context_len,
                                             partition_size))


def pa_decode(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, *,
              max_context_len: int, partition_size: int = 0, workspace: torch.Tensor | None = None,
              status: DeviceStatus | None = None, stream=None, phase: int = 0,
              k_new: torch.Tensor | None = None, v_new: torch.Tensor | None = None,
              slot_mapping: torch.Tensor | None = None, simt: bool = False,
              skip_counter_reset: bool = False) -> torch.Tensor:
    """Paged decode attention; writes ``out`` [S, Hq, hd] and returns it.

    q [S, Hq, hd]; k_cache, v_cache [num_blocks, Hkv, block_size, hd];
    block_tables [S, max_blocks] int32; context_lens [S] int32.  When any
    sequence may span more than one partition a workspace of
    ``pa_decode_workspace_size`` bytes is needed; if none is given one is
    allocated (zeroed) with torch for this call.  ``skip_counter_reset=True``
    skips the reset of the workspace's work counter; valid when the counter is
    zero (a zeroed workspace, or one a completed call has used).

    With k_new, v_new [S, Hkv, hd] and slot_mapping [S] int64, each
    sequence's new (last) token is written into the caches and attended in the
    same launch (fused cache write).  ``simt=True`` (bf16 only) computes the
    products with fp32 FMAs instead of tensor-core MMAs.
    """
    call = _decode_call(out, q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len,
                        partition_size, workspace, status, phase, k_new, v_new, slot_mapping, simt,
                        skip_counter_reset, stream=stream)
    return call(stream)


def pa_decode_window_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                    max_context_len: int, partition_size: int = 0, *, window: int,
                                    num_sinks: int = 0, dtype: torch.dtype = torch.bfloat16) -> int:
    return int(_lib.pa_decode_window_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                                                    partition_size, window, num_sinks, _dtype_code(dtype)))


def pa_decode_window(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, *, window: int,
                     num_sinks: int = 0, max_context_len: int, partition_size: int = 0,
                     workspace: torch.Tensor | None = None, status: DeviceStatus | None = None, stream=None,
                     phase: int = 0, k_new: torch.Tensor | None = None, v_new: torch.Tensor | None = None,
                     slot_mapping: torch.Tensor | None = None, skip_counter_reset: bool = False) -> torch.Tensor:
    """``pa_decode`` over the last ``window`` tokens of each sequence and its
    first ``num_sinks``.  Blocks that hold none of them are not looked up, so
    their table entries may hold anything.  The other arguments are those of
    ``pa_decode``; the workspace takes ``pa_decode_window_workspace_size`` bytes.
    """
    if window < 1 or num_sinks < 0:
        raise ValueError("window must be at least 1 and num_sinks at least 0")
    call = _decode_call(out, q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len,
                        partition_size, workspace, status, phase, k_new, v_new, slot_mapping, False,
                        skip_counter_reset, window, num_sinks, stream)
    return call(stream)


class _PreparedCall:
    """A checked decode call: pointers and sizes are taken from its tensors,
    which it keeps, once; each call enqueues it on a stream."""

    def __init__(self, fn, out, operands, sizes, args, device, keep):
        self._fn, self._out, self._args, self._device, self._keep = fn, out, args, device, keep
        self._operands = [ctypes.c_void_p(t.data_ptr()) for t in (out, *operands)]
        self._sizes, self._ref = sizes, ctypes.byref(args)

    def owns_workspace(self, workspace) -> bool:
        """Whether the call runs on this workspace or none, so that it may be kept:
        one that had a workspace made for it serves the stream it was made on."""
        return not self._args.workspace or workspace is not None

    def __call__(self, stream=None, phase=None) -> torch.Tensor:
        a = self._args
        a.stream = _stream_ptr(stream, self._device)
        if phase is not None:
            a.phase = phase
        _call(self._device, self._fn, *self._operands, *self._sizes, self._ref)
        return self._out


def _decode_call(out, q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len, partition_size,
                 workspace, status, phase, k_new, v_new, slot_mapping, simt, skip_counter_reset, window=0,
                 num_sinks=0, stream=None) -> _PreparedCall:
    """The checks and arguments of pa_decode (window 0) and pa_decode_window."""
    fdt = (torch.float32, torch.bfloat16)
    _check_cuda(q, "q", fdt)
    dev = q.device
    _check_cuda(out, "out", (q.dtype,), dev)
    _check_cuda(k_cache, "k_cache", (q.dtype,), dev)
    _check_cuda(v_cache, "v_cache", (q.dtype,), dev)
    _check_cuda(block_tables, "block_tables", (torch.int32,), dev)
    _check_cuda(context_lens, "context_lens", (torch.int32,), dev)
    if q.dim() != 3 or k_cache.dim() != 4 or block_tables.dim() != 2:
        raise ValueError("q must be [S, Hq, hd], caches [num_blocks, Hkv, bs, hd], tables [S, max_blocks]")
    S, Hq, hd = q.shape
    nb, Hkv, bs, hd2 = k_cache.shape
    if (hd2 != hd or tuple(v_cache.shape) != tuple(k_cache.shape) or tuple(out.shape) != tuple(q.shape)
            or block_tables.shape[0] != S or tuple(context_lens.shape) != (S,)):
        raise ValueError("inconsistent shapes")
    if window:
        need = pa_decode_window_workspace_size(S, Hq, Hkv, hd, max_context_len, partition_size, window=window,
                                               num_sinks=num_sinks, dtype=q.dtype)
    else:
        need = pa_decode_workspace_size(S, Hq, hd, max_context_len, partition_size)
    workspace, skip_counter_reset = _workspace(workspace, need, skip_counter_reset, dev, stream)
    fused = (k_new, v_new, slot_mapping)
    if any(t is not None for t in fused):
        if any(t is None for t in fused):
            raise ValueError("k_new, v_new and slot_mapping go together")
        _check_cuda(k_new, "k_new", (q.dtype,), dev)
        _check_cuda(v_new, "v_new", (q.dtype,), dev)
        _check_cuda(slot_mapping, "slot_mapping", (torch.int64,), dev)
        if tuple(k_new.shape) != (S, Hkv, hd) or tuple(v_new.shape) != (S, Hkv, hd) or \
                tuple(slot_mapping.shape) != (S,):
            raise ValueError("k_new, v_new must be [S, Hkv, hd] and slot_mapping [S]")
    args = _DecodeArgs(S, block_tables.shape[1], nb, _dtype_code(q.dtype), partition_size,
                       max_context_len,
                       workspace.data_ptr() if workspace is not None else None,
                       workspace.numel() if workspace is not None else 0,
                       status.ptr() if status is not None else None,
                       None, phase,
                       k_new.data_ptr() if k_new is not None else None,
                       v_new.data_ptr() if v_new is not None else None,
                       slot_mapping.data_ptr() if slot_mapping is not None else None,
                       1 if simt else 0, 1 if skip_counter_reset else 0)
    sizes = [Hq, Hkv, hd, bs, float(scale)]
    keep = (out, q, k_cache, v_cache, block_tables, context_lens, workspace, status, k_new, v_new, slot_mapping)
    operands = (q, k_cache, v_cache, block_tables, context_lens)
    if window:
        return _PreparedCall(_lib.pa_decode_window, out, operands, [*sizes, window, num_sinks], args, dev, keep)
    return _PreparedCall(_lib.pa_decode, out, operands, sizes, args, dev, keep)


def _torch_stream(stream, dev) -> torch.cuda.Stream:
    """A call's ``stream`` argument (a torch stream, another library's, or a handle) as torch's."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(getattr(stream, "cuda_stream", stream))
    # handle 0 is the default stream, but torch takes it for "no handle given"
    # and wraps a stream of its own pool, which nothing orders with the call
    return torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)


def _workspace(workspace, need, skip_counter_reset, dev, stream, zeroed=True):
    """The caller's workspace, checked, or a zeroed one when one is needed: made
    on the stream that uses it, so that its zeros are there in time and its
    memory is not handed out again before the call is done with it."""
    if need and workspace is None:
        make = torch.zeros if zeroed else torch.empty
        if stream is None:
            return make(need, dtype=torch.uint8, device=dev), True
        with torch.cuda.stream(_torch_stream(stream, dev)):
            return make(need, dtype=torch.uint8, device=dev), True
    if workspace is not None:
        _check_cuda(workspace, "workspace", (torch.uint8,), dev)
    return workspace, skip_counter_reset


def pa_reshape_and_cache(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                         slot_mapping: torch.Tensor, *, status: DeviceStatus | None = None,
                         stream=None) -> None:
    """Write k, v [T, Hkv, hd] into the caches at slot_mapping [T] int64."""
    _check_cuda(k_cache, "k_cache", (torch.float32, torch.bfloat16))
    dev = k_cache.device
    for name, t in (("k", k), ("v", v), ("v_cache", v_cache)):
        _check_cuda(t, name, (k_cache.dtype,), dev)
    _check_cuda(slot_mapping, "slot_mapping", (torch.int64,), dev)
    nb, Hkv, bs, hd = k_cache.shape
    T = slot_mapping.shape[0]
    if tuple(k.shape) != (T, Hkv, hd) or tuple(v.shape) != (T, Hkv, hd) or v_cache.shape != k_cache.shape:
        raise ValueError("inconsistent shapes")
    _call(dev, _lib.pa_reshape_and_cache, k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          slot_mapping.data_ptr(), T, Hkv, hd, bs, nb, _dtype_code(k_cache.dtype),
          status.ptr() if status is not None else None, _stream_ptr(stream, dev))


def pa_copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, src_dst_pairs: torch.Tensor, *,
                   status: DeviceStatus | None = None, stream=None) -> None:
    """Copy whole blocks src -> dst in both caches; src_dst_pairs [P, 2] int64."""
    _check_cuda(k_cache, "k_cache", (torch.float32, torch.bfloat16))
    dev = k_cache.device
    _check_cuda(v_cache, "v_cache", (k_cache.dtype,), dev)
    _check_cuda(src_dst_pairs, "src_dst_pairs", (torch.int64,), dev)
    if src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2 or v_cache.shape != k_cache.shape:
        raise ValueError("inconsistent shapes")
    nb, Hkv, bs, hd = k_cache.shape
    with torch.cuda.device(dev):
        rc = _lib.pa_copy_blocks(k_cache.data_ptr(), v_cache.data_ptr(), src_dst_pairs.data_ptr(),
                                 src_dst_pairs.shape[0], Hkv, hd, bs, nb, _dtype_code(k_cache.dtype),
                                 status.ptr() if status is not None else None,
                                 _stream_ptr(stream, dev))
    _raise(rc)


def pa_swap_blocks(src_k: torch.Tensor, src_v: torch.Tensor, dst_k: torch.Tensor, dst_v: torch.Tensor,
                   src_dst_pairs: torch.Tensor, *, status: DeviceStatus | None = None, stream=None) -> None:
    """Copy whole blocks between two pools of the same geometry, each on the
    GPU or in pinned host memory (swap out / swap in).  src_dst_pairs [P, 2]
    int64, on the GPU or pinned."""
    pools = (("src_k", src_k), ("src_v", src_v), ("dst_k", dst_k), ("dst_v", dst_v))
    for name, t in pools:
        if not isinstance(t, torch.Tensor) or t.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"{name} must be an fp32 or bf16 tensor")
        if not t.is_contiguous() or t.dim() != 4:
            raise ValueError(f"{name} must be a contiguous [num_blocks, Hkv, bs, hd] tensor")
        if t.device.type == "cpu" and not t.is_pinned():
            raise ValueError(f"{name} is pageable host memory; pin it (pin_memory()) so the GPU can address it")
    if src_k.shape[1:] != dst_k.shape[1:] or src_v.shape != src_k.shape or dst_v.shape != dst_k.shape \
            or len({t.dtype for _, t in pools}) != 1:
        raise ValueError("pools must share block geometry and dtype")
    if src_dst_pairs.dtype != torch.int64 or src_dst_pairs.dim() != 2 or src_dst_pairs.shape[1] != 2:
        raise ValueError("src_dst_pairs must be int64 [P, 2]")
    if src_dst_pairs.device.type == "cpu" and not src_dst_pairs.is_pinned():
        raise ValueError("src_dst_pairs must be on the GPU or pinned")
    devs = {t.device for _, t in pools if t.device.type == "cuda"}
    if src_dst_pairs.device.type == "cuda":
        devs.add(src_dst_pairs.device)
    if len(devs) > 1:
        raise ValueError("all device tensors must be on one GPU")
    dev = devs.pop() if devs else torch.device("cuda", torch.cuda.current_device())
    nbs, Hkv, bs, hd = src_k.shape
    with torch.cuda.device(dev):
        rc = _lib.pa_swap_blocks(src_k.data_ptr(), src_v.data_ptr(), dst_k.data_ptr(), dst_v.data_ptr(),
                                 src_dst_pairs.data_ptr(), src_dst_pairs.shape[0], nbs, dst_k.shape[0], Hkv, hd,
                                 bs, _dtype_code(src_k.dtype), status.ptr() if status is not None else None,
                                 _stream_ptr(stream, dev))
    _raise(rc)


def pa_build_tables(block_tables: torch.Tensor, slot_mapping: torch.Tensor, positions: torch.Tensor | None,
                    query_start: torch.Tensor | None, block_ids: torch.Tensor, context_lens: torch.Tensor,
                    new_lens: torch.Tensor, *, block_size: int, num_blocks: int,
                    status: DeviceStatus | None = None, stream=None) -> None:
    """Lay out a batch's tables on the GPU from its lengths and flat block list.

    Inputs (int32, on the GPU): block_ids [N], every sequence's blocks in
    order without padding; context_lens [S], the tokens each sequence holds
    after this step; new_lens [S], how many of them (the last ones) are new.
    Outputs: block_tables [S, max_blocks] int32 padded with -1; slot_mapping
    [T] int64 and positions [T] int32 (or None) of the new tokens, sequence by
    sequence, rows behind the last token -1 and 0; query_start [S + 1] int32
    (or None), where each sequence's new tokens begin.
    ``BlockManager.flat_blocks`` gives block_ids and context_lens.
    """
    _check_cuda(block_tables, "block_tables", (torch.int32,))
    dev = block_tables.device
    _check_cuda(slot_mapping, "slot_mapping", (torch.int64,), dev)
    for name, t in (("block_ids", block_ids), ("context_lens", context_lens), ("new_lens", new_lens)):
        _check_cuda(t, name, (torch.int32,), dev)
    if block_tables.dim() != 2 or slot_mapping.dim() != 1 or block_ids.dim() != 1:
        raise ValueError("block_tables must be [S, max_blocks], slot_mapping [T], block_ids [N]")
    (S, width), T = block_tables.shape, slot_mapping.shape[0]
    if context_lens.shape != (S,) or new_lens.shape != (S,):
        raise ValueError("context_lens and new_lens must be [S]")
    if positions is not None:
        _check_cuda(positions, "positions", (torch.int32,), dev)
        if positions.shape != (T,):
            raise ValueError("positions must be [T] like slot_mapping")
    if query_start is not None:
        _check_cuda(query_start, "query_start", (torch.int32,), dev)
        if query_start.shape != (S + 1,):
            raise ValueError("query_start must be [S + 1]")
    _call(dev, _lib.pa_build_tables, block_tables.data_ptr(), slot_mapping.data_ptr(), _ptr(positions),
          _ptr(query_start), block_ids.data_ptr(), context_lens.data_ptr(), new_lens.data_ptr(), S, width, T,
          block_ids.shape[0], block_size, num_blocks, status.ptr() if status is not None else None,
          _stream_ptr(stream, dev))


def pa_q4_page_bytes(head_dim: int, block_size: int, group_size: int = 64) -> int:
    """Bytes of one page (block, KV head) of a 4-bit cache; its caches are
    uint8 tensors [num_blocks, Hkv, page_bytes]."""
    n = int(_lib.pa_q4_page_bytes(head_dim, block_size, group_size))
    if n == 0:
        raise PAError(PA_ERR_UNSUPPORTED, "pa_q4_page_bytes: head_dim must be 64 or 128, block_size 16 or 32, "
                                          "group_size 32 or 64")
    return n


def q4_block_rows(cache: torch.Tensor, block_size: int) -> torch.Tensor:
    """A 4-bit cache's bytes as the bf16 [num_blocks, Hkv, block_size, n] tensor
    of the same memory that ``pa_copy_blocks`` and ``pa_swap_blocks`` take
    (they move whole blocks bit for bit)."""
    nb, Hkv, page = cache.shape
    if page % (2 * block_size):
        raise ValueError(f"page_bytes {page} does not hold whole rows of {block_size} tokens")
    return cache.view(torch.bfloat16).view(nb, Hkv, block_size, page // (2 * block_size))


def _q4_geometry(k_cache: torch.Tensor, v_cache: torch.Tensor, head_dim: int, group_size: int, dev):
    """Checks a pair of 4-bit caches; returns (num_blocks, Hkv, block_size)."""
    _check_cuda(k_cache, "k_cache", (torch.uint8,), dev)
    _check_cuda(v_cache, "v_cache", (torch.uint8,), dev)
    if k_cache.dim() != 3 or v_cache.shape != k_cache.shape:
        raise ValueError("4-bit caches must be uint8 [num_blocks, Hkv, page_bytes], both of one shape")
    nb, Hkv, page = k_cache.shape
    if head_dim in (64, 128) and group_size in (32, 64):
        bs, rest = divmod(page, head_dim // 2 + 4 * (head_dim // group_size))
        if rest == 0 and bs in (16, 32):
            return nb, Hkv, bs
    raise ValueError(f"page_bytes {page} is not pa_q4_page_bytes({head_dim}, 16 or 32, {group_size})")


def pa_reshape_and_cache_q4(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            slot_mapping: torch.Tensor, *, group_size: int = 64,
                            status: DeviceStatus | None = None, stream=None) -> None:
    """Quantise k, v [T, Hkv, hd] (bf16 or fp32) into the 4-bit caches
    (uint8 [num_blocks, Hkv, page_bytes]) at slot_mapping [T] int64."""
    _q4_rows_call(_lib.pa_reshape_and_cache_q4, k, v, k_cache, v_cache, slot_mapping, group_size, status, stream)


def pa_gather_q4(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 slot_mapping: torch.Tensor, *, group_size: int = 64, status: DeviceStatus | None = None,
                 stream=None) -> None:
    """Read rows of the 4-bit caches back into k, v [T, Hkv, hd] (bf16 or
    fp32); rows with a negative slot are left as they were."""
    _q4_rows_call(_lib.pa_gather_q4, k, v, k_cache, v_cache, slot_mapping, group_size, status, stream)


def pa_decode_q4_workspace_size(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                                max_context_len: int, partition_size: int = 0, *, window: int = 0,
                                num_sinks: int = 0) -> int:
    return int(_lib.pa_decode_q4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, max_context_len,
                                                partition_size, window, num_sinks))


def pa_decode_q4(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 block_tables: torch.Tensor, context_lens: torch.Tensor, scale: float, *, max_context_len: int,
                 group_size: int = 64, window: int = 0, num_sinks: int = 0, partition_size: int = 0,
                 workspace: torch.Tensor | None = None, status: DeviceStatus | None = None, stream=None,
                 phase: int = 0, skip_counter_reset: bool = False) -> torch.Tensor:
    """Paged decode attention over 4-bit caches (uint8 [num_blocks, Hkv,
    page_bytes], written by ``pa_reshape_and_cache_q4``); writes ``out``
    [S, Hq, hd], of q's type, and returns it.

    window 0 attends to every token; otherwise to the last ``window`` tokens
    and the first ``num_sinks``, as ``pa_decode_window`` does.  The workspace,
    where one is needed, takes ``pa_decode_q4_workspace_size`` bytes; the other
    arguments are those of ``pa_decode``.
    """
    return _decode_q4_call(out, q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len, group_size,
                           window, num_sinks, partition_size, workspace, status, phase, skip_counter_reset,
                           stream)(stream)


def _decode_q4_call(out, q, k_cache, v_cache, block_tables, context_lens, scale, max_context_len, group_size,
                    window, num_sinks, partition_size, workspace, status, phase, skip_counter_reset,
                    stream=None) -> _PreparedCall:
    """The checks and arguments of pa_decode_q4."""
    _check_cuda(q, "q", (torch.float32, torch.bfloat16))
    dev = q.device
    _check_cuda(out, "out", (q.dtype,), dev)
    _check_cuda(block_tables, "block_tables", (torch.int32,), dev)
    _check_cuda(context_lens, "context_lens", (torch.int32,), dev)
    if q.dim() != 3 or block_tables.dim() != 2:
        raise ValueError("q must be [S, Hq, hd], tables [S, max_blocks]")
    S, Hq, hd = q.shape
    nb, Hkv, bs = _q4_geometry(k_cache, v_cache, hd, group_size, dev)
    if tuple(out.shape) != tuple(q.shape) or block_tables.shape[0] != S or tuple(context_lens.shape) != (S,):
        raise ValueError("inconsistent shapes")
    need = pa_decode_q4_workspace_size(S, Hq, Hkv, hd, max_context_len, partition_size, window=window,
                                       num_sinks=num_sinks)
    workspace, skip_counter_reset = _workspace(workspace, need, skip_counter_reset, dev, stream)
    args = _DecodeArgs(S, block_tables.shape[1], nb, _dtype_code(q.dtype), partition_size, max_context_len,
                       _ptr(workspace), workspace.numel() if workspace is not None else 0,
                       status.ptr() if status is not None else None, None, phase, None, None, None, 0,
                       1 if skip_counter_reset else 0)
    return _PreparedCall(_lib.pa_decode_q4, out, (q, k_cache, v_cache, block_tables, context_lens),
                         [Hq, Hkv, hd, bs, group_size, float(scale), window, num_sinks], args, dev,
                         (workspace, status, q, k_cache, v_cache, block_tables, context_lens))


def _q4_rows_call(fn, k, v, k_cache, v_cache, slot_mapping, group_size, status, stream):
    _check_cuda(k, "k", (torch.float32, torch.bfloat16))
    dev = k.device
    _check_cuda(v, "v", (k.dtype,), dev)
    _check_cuda(slot_mapping, "slot_mapping", (torch.int64,), dev)
    if k.dim() != 3 or v.shape != k.shape or slot_mapping.shape != (k.shape[0],):
        raise ValueError("k, v must be [T, Hkv, hd] and slot_mapping [T]")
    T, Hkv, hd = k.shape
    nb, heads, bs = _q4_geometry(k_cache, v_cache, hd, group_size, dev)
    if heads != Hkv:
        raise ValueError("inconsistent shapes")
    _call(dev, fn, k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), slot_mapping.data_ptr(), T,
          Hkv, hd, bs, group_size, nb, _dtype_code(k.dtype), status.ptr() if status is not None else None,
          _stream_ptr(stream, dev))


def pa_decode_tree_workspace_size(num_tokens: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(_lib.pa_decode_tree_workspace_size(num_tokens, num_q_heads, num_kv_heads, head_dim))


def pa_decode_tree(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_tables: torch.Tensor, context_lens: torch.Tensor, query_start: torch.Tensor, scale: float, *,
                   max_context_len: int, max_query_len: int = 0, tree_mask: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, status: DeviceStatus | None = None,
                   stream=None) -> torch.Tensor:
    """Attention of drafted tokens over the paged cache; writes ``out``
    [T, Hq, hd] and returns it.

    The rows of q [T, Hq, hd] from query_start[i] (int32 [S + 1]) on are the last
    tokens of sequence i, whose K/V the cache holds already.  Each sees every
    position before the sequence's drafted tokens, and of those the ones whose
    bits are set in its row of tree_mask (int64 [T, W], bit j % 64 of word j // 64;
    ``pa_build_tree`` makes it), or without one those up to itself.  Rows behind
    the last sequence's are left as they were.  The workspace takes
    ``pa_decode_tree_workspace_size`` bytes, whatever the contexts; the other
    arguments are those of ``pa_decode``.

    max_query_len, an upper bound of a sequence's rows (0: unknown), decides which
    kernels run, never what they compute: give it where sequences differ in
    their rows or q has padding.
    """
    return _multi_call(True, out, q, k_cache, v_cache, block_tables, context_lens, query_start, tree_mask, scale,
                       max_context_len, workspace, status, stream, max_query_len)(stream)


def pa_decode_cross(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    block_tables: torch.Tensor, context_lens: torch.Tensor, query_start: torch.Tensor, scale: float,
                    *, max_context_len: int, max_query_len: int = 0, workspace: torch.Tensor | None = None,
                    status: DeviceStatus | None = None, stream=None) -> torch.Tensor:
    """Attention of any number of queries per request over the paged states of
    another sequence (an encoder's): every row of q [T, Hq, hd] from
    query_start[i] on sees all context_lens[i] tokens of block_tables[i].  The
    arguments are those of ``pa_decode_tree``."""
    return _multi_call(False, out, q, k_cache, v_cache, block_tables, context_lens, query_start, None, scale,
                       max_context_len, workspace, status, stream, max_query_len)(stream)


def _multi_call(tree, out, q, k_cache, v_cache, block_tables, context_lens, query_start, tree_mask, scale,
                max_context_len, workspace, status, stream=None, max_query_len=0) -> _PreparedCall:
    """The checks and arguments of pa_decode_tree and pa_decode_cross."""
    _check_cuda(q, "q", (torch.float32, torch.bfloat16))
    dev = q.device
    for name, t in (("out", out), ("k_cache", k_cache), ("v_cache", v_cache)):
        _check_cuda(t, name, (q.dtype,), dev)
    _check_int32(dev, block_tables=block_tables, context_lens=context_lens, query_start=query_start)
    if q.dim() != 3 or k_cache.dim() != 4 or block_tables.dim() != 2:
        raise ValueError("q must be [T, Hq, hd], caches [num_blocks, Hkv, bs, hd], tables [S, max_blocks]")
    T, Hq, hd = q.shape
    nb, Hkv, bs, hd2 = k_cache.shape
    S = block_tables.shape[0]
    if (hd2 != hd or v_cache.shape != k_cache.shape or out.shape != q.shape or context_lens.shape != (S,)
            or query_start.shape != (S + 1,)):
        raise ValueError("inconsistent shapes")
    words = 0
    if tree_mask is not None:
        _check_cuda(tree_mask, "tree_mask", (torch.int64,), dev)
        if tree_mask.dim() != 2 or tree_mask.shape[0] != T:
            raise ValueError("tree_mask must be [T, words]")
        words = tree_mask.shape[1]
    workspace, _ = _workspace(workspace, pa_decode_tree_workspace_size(T, Hq, Hkv, hd), False, dev, stream,
                              zeroed=False)
    args = _DecodeArgs(S, block_tables.shape[1], nb, _dtype_code(q.dtype), 0, max_context_len, _ptr(workspace),
                       workspace.numel() if workspace is not None else 0, status.ptr() if status is not None else None,
                       max_query_len=max_query_len)
    operands = (q, k_cache, v_cache, block_tables, context_lens, query_start)
    sizes = [Hq, Hkv, hd, bs, float(scale), T]
    keep = (workspace, status, tree_mask, *operands)
    if not tree:
        return _PreparedCall(_lib.pa_decode_cross, out, operands, sizes, args, dev, keep)
    return _PreparedCall(_lib.pa_decode_tree, out, operands, [_ptr(tree_mask), *sizes, words], args, dev, keep)


def pa_build_tree(tree_mask: torch.Tensor, positions: torch.Tensor | None, parents: torch.Tensor,
                  query_start: torch.Tensor, context_lens: torch.Tensor, *, status: DeviceStatus | None = None,
                  stream=None) -> None:
    """Ancestor bits and positions of the batch's trees of drafted tokens.

    parents int32 [T]: each node's parent within its tree, an earlier node or -1;
    query_start int32 [S + 1] and context_lens int32 [S] as for ``pa_decode_tree``.
    Writes tree_mask int64 [T, W] (trees of up to 64 W nodes, W <= 16) and
    positions int32 [T] (or None): the sequence's length before its tree plus the
    node's depth.
    """
    _check_cuda(tree_mask, "tree_mask", (torch.int64,))
    dev = tree_mask.device
    _check_int32(dev, parents=parents, query_start=query_start, context_lens=context_lens)
    if positions is not None:
        _check_int32(dev, positions=positions)
    T, S = parents.shape[0], context_lens.shape[0]
    if (tree_mask.dim() != 2 or tree_mask.shape[0] != T or parents.shape != (T,) or context_lens.shape != (S,)
            or query_start.shape != (S + 1,) or (positions is not None and positions.shape != (T,))):
        raise ValueError("tree_mask must be [T, words], parents and positions [T], context_lens [S], "
                         "query_start [S + 1]")
    _call(dev, _lib.pa_build_tree, tree_mask.data_ptr(), _ptr(positions), parents.data_ptr(), query_start.data_ptr(),
          context_lens.data_ptr(), S, T, tree_mask.shape[1], status.ptr() if status is not None else None,
          _stream_ptr(stream, dev))


def pa_accept_tree(accepted_lens: torch.Tensor, accepted_nodes: torch.Tensor, next_tokens: torch.Tensor,
                   new_lens: torch.Tensor, slot_pairs: torch.Tensor, draft_tokens: torch.Tensor,
                   target_tokens: torch.Tensor, parents: torch.Tensor | None, query_start: torch.Tensor,
                   context_lens: torch.Tensor, block_tables: torch.Tensor, *, block_size: int, num_blocks: int,
                   status: DeviceStatus | None = None, stream=None) -> None:
    """The path of each tree that the target model agrees with.

    draft_tokens int32 [T]: the nodes' tokens; target_tokens int32 [T]: the target
    model's choice behind each node; parents as for ``pa_build_tree``, None for
    chains.  Node 0 is always accepted, then the lowest child whose token is the
    target's choice, up to M = accepted_nodes.shape[1] nodes.  Writes, int32 and
    per sequence, accepted_lens [S], accepted_nodes [S, M] (-1 behind the path),
    next_tokens [S] (the target's choice at the path's end) and new_lens [S], and
    slot_pairs int64 [S, M, 2], the (source, destination) slots by which
    ``pa_move_rows`` puts the path's rows where the sequence goes on.
    """
    _check_cuda(accepted_nodes, "accepted_nodes", (torch.int32,))
    dev = accepted_nodes.device
    _check_int32(dev, accepted_lens=accepted_lens, next_tokens=next_tokens, new_lens=new_lens,
                 draft_tokens=draft_tokens, target_tokens=target_tokens, query_start=query_start,
                 context_lens=context_lens, block_tables=block_tables)
    _check_cuda(slot_pairs, "slot_pairs", (torch.int64,), dev)
    if parents is not None:
        _check_int32(dev, parents=parents)
    if accepted_nodes.dim() != 2 or block_tables.dim() != 2 or draft_tokens.dim() != 1:
        raise ValueError("accepted_nodes must be [S, M], block_tables [S, max_blocks], draft_tokens [T]")
    (S, M), T = accepted_nodes.shape, draft_tokens.shape[0]
    if (accepted_lens.shape != (S,) or next_tokens.shape != (S,) or new_lens.shape != (S,)
            or context_lens.shape != (S,) or slot_pairs.shape != (S, M, 2) or target_tokens.shape != (T,) or query_start.shape != (S + 1,)
            or block_tables.shape[0] != S or (parents is not None and parents.shape != (T,))):
        raise ValueError("inconsistent shapes")
    _call(dev, _lib.pa_accept_tree, accepted_lens.data_ptr(), accepted_nodes.data_ptr(), next_tokens.data_ptr(),
          new_lens.data_ptr(), slot_pairs.data_ptr(), draft_tokens.data_ptr(), target_tokens.data_ptr(),
          _ptr(parents), query_start.data_ptr(), context_lens.data_ptr(), block_tables.data_ptr(), S, T, M,
          block_tables.shape[1], block_size, num_blocks, status.ptr() if status is not None else None,
          _stream_ptr(stream, dev))


MOVE_GROUP_BYTES = 48 * 1024   # of one head's rows in a group of pa_move_rows


def pa_move_rows(k_cache: torch.Tensor, v_cache: torch.Tensor, slot_pairs: torch.Tensor, *,
                 status: DeviceStatus | None = None, stream=None) -> None:
    """Move K/V rows from slot to slot, every KV head: slot_pairs int64
    [groups, pairs, 2] (source, destination), negative ones skipped.  Within a
    group every source is read before any destination is written, and its rows
    of one head fit in ``MOVE_GROUP_BYTES`` (``TreeDecodeStep.commit`` takes
    longer paths)."""
    _check_cuda(k_cache, "k_cache", (torch.float32, torch.bfloat16))
    dev = k_cache.device
    _check_cuda(v_cache, "v_cache", (k_cache.dtype,), dev)
    _check_cuda(slot_pairs, "slot_pairs", (torch.int64,), dev)
    if slot_pairs.dim() != 3 or slot_pairs.shape[2] != 2 or k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("slot_pairs must be [groups, pairs, 2], caches [num_blocks, Hkv, bs, hd]")
    nb, Hkv, bs, hd = k_cache.shape
    _call(dev, _lib.pa_move_rows, k_cache.data_ptr(), v_cache.data_ptr(), slot_pairs.data_ptr(), slot_pairs.shape[0],
          slot_pairs.shape[1], Hkv, hd, bs, nb, _dtype_code(k_cache.dtype),
          status.ptr() if status is not None else None, _stream_ptr(stream, dev))


class BlockManager:
    """Host block manager (``pa_bm_*``): free pool, refcounts, copy-on-write."""

    def __init__(self, num_blocks: int, block_size: int):
        self._h = _lib.pa_bm_create(num_blocks, block_size)
        if not self._h:
            raise PAError(PA_ERR_INVALID_ARG, _lib.pa_last_error_string().decode())
        self.num_blocks = num_blocks
        self.block_size = block_size

    def close(self):
        if self._h:
            _lib.pa_bm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add_seq(self, seq_id: int, num_tokens: int) -> None:
        _raise(_lib.pa_bm_add_seq(self._h, seq_id, num_tokens))

    def fork(self, parent: int, child: int) -> None:
        _raise(_lib.pa_bm_fork(self._h, parent, child))

    def append_slot(self, seq_id: int):
        slot = ctypes.c_int64()
        src, dst = ctypes.c_int32(), ctypes.c_int32()
        _raise(_lib.pa_bm_append_slot(self._h, seq_id, ctypes.byref(slot), ctypes.byref(src),
                                      ctypes.byref(dst)))
        return slot.value, src.value, dst.value

    def append_slots(self, seq_ids):
        """Batched append; returns (slots int64 [n], cow_pairs int64 [P, 2])."""
        ids = torch.tensor(list(seq_ids), dtype=torch.int32)
        n = ids.numel()
        slots = torch.empty(n, dtype=torch.int64)
        pairs = torch.empty(max(n, 1), 2, dtype=torch.int64)
        npairs, ndone = ctypes.c_int(), ctypes.c_int()
        rc = _lib.pa_bm_append_slots(self._h, ids.data_ptr(), n, slots.data_ptr(), pairs.data_ptr(),
                                     ctypes.byref(npairs), ctypes.byref(ndone))
        _raise(rc)
        return slots, pairs[:npairs.value].clone()

    def add_seq_cached(self, seq_id: int, tokens, salt: int = 0) -> int:
        """New sequence over token ids, sharing cached prefix blocks (chained
        block keys, tenant salt).  Returns the number of leading tokens whose
        K/V are already in the cache."""
        t = torch.as_tensor(list(tokens) if not isinstance(tokens, torch.Tensor) else tokens,
                            dtype=torch.int32).contiguous()
        cached = ctypes.c_int()
        _raise(_lib.pa_bm_add_seq_cached(self._h, seq_id, t.data_ptr() if t.numel() else None, t.numel(),
                                         ctypes.c_uint64(salt & (2**64 - 1)), ctypes.byref(cached)))
        return cached.value

    def register_blocks(self, seq_id: int, tokens, salt: int = 0) -> int:
        """Key the sequence's full blocks not keyed yet; returns how many."""
        t = torch.as_tensor(list(tokens) if not isinstance(tokens, torch.Tensor) else tokens,
                            dtype=torch.int32).contiguous()
        n = _lib.pa_bm_register_blocks(self._h, seq_id, t.data_ptr() if t.numel() else None, t.numel(),
                                       ctypes.c_uint64(salt & (2**64 - 1)))
        if n < 0:
            _raise(n)
        return n

    def num_cached(self) -> int:
        return _lib.pa_bm_num_cached(self._h)

    def move_seq(self, to: "BlockManager", seq_id: int) -> torch.Tensor:
        """Move a sequence into another manager's pool; returns the int64
        [P, 2] (block here, block there) pairs for pa_swap_blocks."""
        cap = max(1, len(self.block_table(seq_id)))
        pairs = torch.empty(cap, 2, dtype=torch.int64)
        n = ctypes.c_int()
        _raise(_lib.pa_bm_move_seq(self._h, to._h, seq_id, pairs.data_ptr(), cap, ctypes.byref(n)))
        return pairs[:n.value].clone()

    def free_seq(self, seq_id: int) -> None:
        _raise(_lib.pa_bm_free_seq(self._h, seq_id))

    def trim_seq(self, seq_id: int, num_tokens: int) -> None:
        """Keep the sequence's first tokens only; blocks past them are released."""
        _raise(_lib.pa_bm_trim_seq(self._h, seq_id, num_tokens))

    def block_table(self, seq_id: int) -> list[int]:
        cap = max(1, self.num_blocks)
        buf = (ctypes.c_int32 * cap)()
        n = _lib.pa_bm_block_table(self._h, seq_id, buf, cap)
        if n < 0:
            _raise(n)
        return list(buf[:n])

    def num_tokens(self, seq_id: int) -> int:
        n = _lib.pa_bm_num_tokens(self._h, seq_id)
        if n < 0:
            _raise(n)
        return n

    def num_free(self) -> int:
        return _lib.pa_bm_num_free(self._h)

    def refcount(self, block: int) -> int:
        r = _lib.pa_bm_refcount(self._h, block)
        if r < 0:
            _raise(r)
        return r

    def flat_blocks(self, seq_ids):
        """Block ids of a batch without padding, int32 [N], and context
        lengths, int32 [n] (host): what ``pa_build_tables`` lays out."""
        ids = torch.tensor(list(seq_ids), dtype=torch.int32)
        n = ids.numel()
        lens = torch.tensor([self.num_tokens(s) for s in ids.tolist()], dtype=torch.int32)
        cap = int(((lens.long() + self.block_size - 1) // self.block_size).sum())
        out = torch.empty(cap, dtype=torch.int32)
        got = _lib.pa_bm_flat_blocks(self._h, ids.data_ptr() if n else None, n, out.data_ptr() if cap else None, cap,
                                     lens.data_ptr() if n else None)
        if got < 0:
            _raise(got)
        return out[:got], lens

    def build_tables(self, seq_ids, max_blocks_per_seq: int):
        """Padded int32 tables [n, max_blocks_per_seq] and context lengths [n] (host)."""
        ids = torch.tensor(list(seq_ids), dtype=torch.int32)
        n = ids.numel()
        tables = torch.empty(n, max_blocks_per_seq, dtype=torch.int32)
        lens = torch.empty(n, dtype=torch.int32)
        _raise(_lib.pa_bm_build_tables(self._h, ids.data_ptr(), n, tables.data_ptr(),
                                       max_blocks_per_seq, lens.data_ptr()))
        return tables, lens
