"""Python binding of libpa.so: paged varlen attention for GB300 (sm_103a).

Thin ctypes marshalling over the C ABI in include/pa.h. Torch is used for
device memory (outputs and workspaces are allocated here, on the caller's
side of the ABI) and for the current CUDA stream; every step of the
computation runs in the library's CUDA kernels. There is no CPU fallback: the
functions raise if the library or a GPU is missing.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libpa.so")

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_BLOCK_SIZE = 2
PA_ERR_UNSUPPORTED = 3
PA_ERR_WORKSPACE = 4
PA_ERR_CUDA = 5
PA_ERR_NOALLOC_LIMIT = 6
NOALLOC_SCRATCH_BYTES = 32 << 20
PA_DEV_BAD_PAGE = 1
PA_DEV_BAD_SLOT = 2
PA_DEV_BAD_SEQLEN = 4
PA_DEV_TIMEOUT = 8
PA_DEV_CASCADE = 16
PA_DEV_BAD_POSITION = 32
PA_BF16 = 0
PA_F16 = 1
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "wavelength": 3, "yarn": 4}

EXPORTS = (
    "pa_status_string",
    "pa_abi_version",
    "pa_reshape_and_cache",
    "pa_varlen_fwd_workspace_size",
    "pa_varlen_fwd",
    "pa_merge_attn_states",
    "pa_cascade_fwd_workspace_size",
    "pa_cascade_fwd",
    "pa_varlen_fwd_noalloc",
    "pa_varlen_fwd_with_update",
    "pa_cascade_fwd_with_update",
    "pa_use_cascade_attention",
    "pa_reshape_and_cache_fp8",
    "pa_varlen_fwd_fp8kv_workspace_size",
    "pa_cascade_fwd_fp8kv_workspace_size",
    "pa_varlen_fwd_fp8kv",
    "pa_cascade_fwd_fp8kv",
    "pa_merge_attn_states_n",
    "pa_varlen_fwd_ex",
    "pa_cascade_fwd_ex",
    "pa_window_fwd",
    "pa_rope_table",
    "pa_rope_and_cache",
    "pa_attn_weights",
    "pa_evict",
)

_lib = None

_c = ctypes
_vp, _i64, _i32, _f32, _sz = _c.c_void_p, _c.c_int64, _c.c_int, _c.c_float, _c.c_size_t
_f64 = _c.c_double
_INT_MAX = 0x7fffffff


class KvUpdate(ctypes.Structure):
    """struct pa_kv_update of include/pa.h."""
    _fields_ = [("key", _vp), ("value", _vp), ("key_token_stride", _i64),
                ("value_token_stride", _i64), ("slot_mapping", _vp), ("num_tokens", _i32)]


class KvFp8(ctypes.Structure):
    """struct pa_kv_fp8 of include/pa.h (device float32 [num_kv_heads] scales)."""
    _fields_ = [("k_scale", _vp), ("v_scale", _vp)]


class AttnOpts(ctypes.Structure):
    """struct pa_attn_opts of include/pa.h."""
    _fields_ = [("sinks", _vp), ("fp8", ctypes.POINTER(KvFp8))]


class RopeScaling(ctypes.Structure):
    """struct pa_rope_scaling of include/pa.h."""
    _fields_ = [("kind", _i32), ("factor", _f64), ("orig_len", _f64), ("low", _f64),
                ("high", _f64), ("mscale", _f64)]


class Rope(ctypes.Structure):
    """struct pa_rope of include/pa.h."""
    _fields_ = [("cos_sin", _vp), ("table_len", _i32), ("rot_dim", _i32), ("interleaved", _i32),
                ("q_norm", _vp), ("k_norm", _vp), ("norm_eps", _f32)]


_ATTN_ARGS = [_vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32,
              _i32, _i32, _i32, _f32, _i32, _vp, _vp, _vp, _sz, _i32, _vp, _vp]

_SIGS = {
    "pa_status_string": ([_i32], _c.c_char_p),
    "pa_abi_version": ([], _i32),
    "pa_reshape_and_cache": ([_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i32, _i32, _i32, _i32,
                              _i32, _i32, _vp, _vp], _i32),
    "pa_varlen_fwd_workspace_size": ([_i32] * 9, _sz),
    "pa_varlen_fwd": ([_vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                       _i32, _i32, _i32, _i32, _i32, _f32, _i32, _vp, _vp, _vp, _sz, _i32, _vp,
                       _vp], _i32),
    "pa_merge_attn_states": ([_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp], _i32),
    "pa_cascade_fwd_workspace_size": ([_i32] * 9, _sz),
    "pa_varlen_fwd_noalloc": ([_vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                               _i32, _i32, _i32, _i32, _i32, _i32, _f32, _i32, _vp, _vp, _i32, _vp,
                               _vp], _i32),
    "pa_cascade_fwd": ([_vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                        _i32, _i32, _i32, _i32, _i32, _f32, _i32, _vp, _vp, _vp, _sz, _i32, _vp,
                        _vp], _i32),
    "pa_varlen_fwd_with_update": ([ctypes.POINTER(KvUpdate)] + _ATTN_ARGS, _i32),
    "pa_cascade_fwd_with_update": ([ctypes.POINTER(KvUpdate)] + _ATTN_ARGS, _i32),
    "pa_use_cascade_attention": ([_i32, _i32, _i32, _i32, _i32, ctypes.POINTER(_i32)], _i32),
    "pa_reshape_and_cache_fp8": ([_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i32, _i32, _i32,
                                  _i32, _i32, ctypes.POINTER(KvFp8), _i32, _vp, _vp], _i32),
    "pa_varlen_fwd_fp8kv_workspace_size": ([_i32] * 9, _sz),
    "pa_merge_attn_states_n": ([_vp, _vp, _vp, _i64, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _vp],
                               _i32),
    "pa_varlen_fwd_ex": ([ctypes.POINTER(KvUpdate)] + _ATTN_ARGS[:20] +
                         [ctypes.POINTER(AttnOpts)] + _ATTN_ARGS[20:], _i32),
    "pa_cascade_fwd_ex": ([ctypes.POINTER(KvUpdate)] + _ATTN_ARGS[:20] +
                          [ctypes.POINTER(AttnOpts)] + _ATTN_ARGS[20:], _i32),
    "pa_window_fwd": ([ctypes.POINTER(KvUpdate)] + _ATTN_ARGS[:20] +
                      [_i32, ctypes.POINTER(AttnOpts)] + _ATTN_ARGS[20:], _i32),
    "pa_rope_table": ([_vp, _i32, _i32, _f64, ctypes.POINTER(RopeScaling), _vp], _i32),
    "pa_rope_and_cache": ([ctypes.POINTER(Rope), _vp, _vp, _i64, _vp, _i64,
                           ctypes.POINTER(KvUpdate), _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32,
                           ctypes.POINTER(KvFp8), _i32, _vp, _vp], _i32),
    "pa_attn_weights": ([_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp] + [_i32] * 10 + [
        _f32, _i32, _vp, _i64, ctypes.POINTER(KvFp8), _i32, _vp, _vp], _i32),
    "pa_evict": ([_vp, _vp, _i64, _vp, _i64, _vp, _vp] + [_i32] * 11 + [_vp, _vp, _vp, _vp],
                 _i32),
    "pa_cascade_fwd_fp8kv_workspace_size": ([_i32] * 9, _sz),
    "pa_varlen_fwd_fp8kv": ([ctypes.POINTER(KvUpdate)] + _ATTN_ARGS[:20] +
                            [ctypes.POINTER(KvFp8)] + _ATTN_ARGS[20:], _i32),
    "pa_cascade_fwd_fp8kv": ([ctypes.POINTER(KvUpdate)] + _ATTN_ARGS[:20] +
                             [ctypes.POINTER(KvFp8)] + _ATTN_ARGS[20:], _i32),
}


def load_library(path: str = LIB_PATH):
    """Load libpa.so (built by ``_build.build()``) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libpa.so not built ({path}); run __graft_entry__.build() "
                           "or python paged_kv_varlen_attn_gb300/_build.py")
    lib = ctypes.CDLL(path)
    for name, (args, res) in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


class PAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = load_library().pa_status_string(code).decode()
        super().__init__(f"{where}: {msg}")


def _check(code: int, where: str):
    if code != PA_OK:
        raise PAError(code, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


def _call(fn, where, device, *args):
    """Call an entry point whose last argument is the stream, on the tensors'
    device (entered only if it is not the current one)."""
    index = device.index
    if index == torch._C._cuda_getDevice():
        code = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            code = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if code != PA_OK:
        raise PAError(code, where)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")


def _one_device(first, *rest):
    """All tensors (None aside) are on the first one's GPU."""
    index = first.get_device()
    if index < 0:
        raise ValueError("all tensors must be CUDA tensors (no CPU fallback)")
    for t in rest:
        if t is not None and t.get_device() != index:
            raise ValueError("all tensors must be on one GPU (no CPU fallback)")


def _fit32(*values):
    """Refuse integers that the C interface does not hold (ctypes would pass
    their low 32 bits on). Called where one may be such: v >> 31 is not 0."""
    for v in values:
        if v > _INT_MAX or v < -_INT_MAX:
            raise ValueError(f"integer arguments must fit 32 bits, got {v}")


def _pools(key_cache, value_cache):
    """(shape, page stride) of a pair of pools laid out alike."""
    shape, st = key_cache.shape, key_cache.stride()
    if st != value_cache.stride() or shape != value_cache.shape:
        raise ValueError("key and value caches must have the same shape and page stride")
    if len(st) == 4:
        _, _, heads, dim = shape
        if st[3] == 1 and st[2] == dim and st[1] == heads * dim:
            return shape, st[0]
    raise ValueError("cache must be [num_blocks, block_size, num_kv_heads, head_size] with "
                     "contiguous pages")


def _seq_table(seqused_k, block_table, num_seqs):
    """Row stride of a block table [num_seqs, columns], which stands for its
    columns: a row may be read up to it."""
    if seqused_k.dtype is not torch.int32 or seqused_k.shape != (num_seqs,) or \
            not seqused_k.is_contiguous():
        raise ValueError("seqused_k must be a contiguous int32 tensor of one value per sequence")
    shape = block_table.shape
    if block_table.dtype is not torch.int32 or len(shape) != 2 or shape[0] != num_seqs:
        raise ValueError("block_table must be int32 [num_seqs, max_blocks]")
    width = shape[1]
    row, unit = block_table.stride()
    if width > 1 and unit != 1:
        raise ValueError("block_table must have unit column stride")
    if row != width and num_seqs > 1:
        end = block_table.storage_offset() + num_seqs * row
        if row < width or end * 4 > block_table.untyped_storage().nbytes():
            raise ValueError("block_table rows must not overlap, and its last row must be followed "
                             "by the rest of a row stride")
        return row
    return width


def _dtype_code(*ts):
    """PA_BF16 or PA_F16 for tensors that must all share one 2-byte float type."""
    dt = ts[0].dtype
    for t in ts:
        if t is not None and t.dtype is not dt:
            names = sorted({str(t.dtype) for t in ts if t is not None})
            raise ValueError(f"tensors must share one element type, got {names}")
    if dt == torch.bfloat16:
        return PA_BF16
    if dt == torch.float16:
        return PA_F16
    raise ValueError(f"unsupported element type {dt} (bfloat16 or float16)")


def _sm_count(device) -> int:
    return torch.cuda.get_device_properties(device).multi_processor_count


def _row_stride(t):
    """Token stride of a [T, heads, D] tensor whose [heads, D] rows are contiguous."""
    st = t.stride()
    if len(st) != 3 or st[2] != 1 or st[1] != t.shape[2]:
        raise ValueError("tensor must be [tokens, heads, head_size] with contiguous rows")
    return st[0]


def _cache_stride(c):
    st = c.stride()
    if len(st) == 4:
        _, _, heads, dim = c.shape
        if st[3] == 1 and st[2] == dim and st[1] == heads * dim:
            return st[0]
    raise ValueError("cache must be [num_blocks, block_size, num_kv_heads, head_size] with "
                     "contiguous pages")


# ---------------------------------------------------------------------------
def reshape_and_cache(key, value, key_cache, value_cache, slot_mapping, dev_status=None):
    """Scatter new K/V rows into their pages (in place on the caches)."""
    lib = load_library()
    _need_cuda(key, value, key_cache, value_cache, slot_mapping, dev_status)
    if key_cache.stride(0) != value_cache.stride(0):
        raise ValueError("key and value caches must share the page stride")
    nb, bs, hk, d = key_cache.shape
    dtype = _dtype_code(key, value, key_cache, value_cache)
    code = lib.pa_reshape_and_cache(
        _ptr(key), _ptr(value), _row_stride(key), _row_stride(value), _ptr(key_cache),
        _ptr(value_cache), _cache_stride(key_cache), _ptr(slot_mapping), key.shape[0], hk, d, bs,
        nb, dtype, _ptr(dev_status), _stream(key.device))
    _check(code, "pa_reshape_and_cache")


def varlen_fwd_workspace_size(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads,
                              num_kv_heads, head_size, block_size, sm_count):
    return load_library().pa_varlen_fwd_workspace_size(
        num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_size,
        block_size, sm_count)


def cascade_fwd_workspace_size(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads,
                               num_kv_heads, head_size, block_size, sm_count):
    return load_library().pa_cascade_fwd_workspace_size(
        num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_size,
        block_size, sm_count)


def use_cascade_attention(common_prefix_len, num_seqs, num_kv_heads, head_size, split_kv=True):
    """Whether a batch whose sequences share common_prefix_len tokens should
    run as cascade attention (host-side policy, no GPU needed)."""
    out = _i32(0)
    _check(load_library().pa_use_cascade_attention(int(common_prefix_len), int(num_seqs),
                                                   int(num_kv_heads), int(head_size),
                                                   int(bool(split_kv)), ctypes.byref(out)),
           "pa_use_cascade_attention")
    return bool(out.value)


def alloc_workspace(nbytes, device):
    # 256-byte aligned (the caching allocator aligns to 512 bytes).
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _attn_common(q, key_cache, value_cache, cu_seqlens_q, seqused_k, block_table):
    _need_cuda(q, key_cache, value_cache, cu_seqlens_q, seqused_k, block_table)
    if key_cache.stride(0) != value_cache.stride(0) or key_cache.shape != value_cache.shape:
        raise ValueError("key and value caches must have the same shape and page stride")
    for t, name in ((cu_seqlens_q, "cu_seqlens_q"), (seqused_k, "seqused_k"),
                    (block_table, "block_table")):
        if t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
    if block_table.dim() != 2 or block_table.stride(1) != 1:
        raise ValueError("block_table must be [num_seqs, max_blocks] with unit column stride")


def _kv_update(key, value, slot_mapping):
    if key is None:
        return None
    _need_cuda(key, value, slot_mapping)
    return KvUpdate(key.data_ptr(), value.data_ptr(), _row_stride(key), _row_stride(value),
                    slot_mapping.data_ptr(), key.shape[0])


def _attend(entry, update, q, key_cache, value_cache, cu_seqlens_q, seqused_k, block_table,
            max_seqlen_q, max_seqlen_k, softmax_scale, mode_arg, out, lse, return_lse,
            workspace, dev_status, size_fn, fp8=None, sinks=None, update_tensors=None):
    lib = load_library()
    _attn_common(q, key_cache, value_cache, cu_seqlens_q, seqused_k, block_table)
    T, H, D = q.shape
    nb, bs, hk, _ = key_cache.shape
    S = cu_seqlens_q.numel() - 1
    if out is None:
        out = torch.empty((T, H, D), dtype=q.dtype, device=q.device)
    # q, out, the new tokens and (unless they hold e4m3 bytes) the pools share the type
    pools = () if fp8 is not None else (key_cache, value_cache)
    dtype = _dtype_code(q, out, *pools, *((update_tensors or ()) if update is not None else ()))
    if lse is None and return_lse:
        lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(size_fn(S, T, max_seqlen_q, max_seqlen_k, H, hk, D, bs,
                                            _sm_count(q.device)), q.device)
    args = (_ptr(q), _row_stride(q), _ptr(key_cache), _ptr(value_cache), _cache_stride(key_cache),
            _ptr(cu_seqlens_q), _ptr(seqused_k), _ptr(block_table), block_table.stride(0), S, T,
            int(max_seqlen_q), int(max_seqlen_k), H, hk, D, bs, nb, float(softmax_scale),
            int(mode_arg)) + ((ctypes.byref(fp8),) if fp8 is not None else ()) + (
            _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(), dtype,
            _ptr(dev_status), _stream(q.device))
    upd = ctypes.byref(update) if update is not None else None
    if sinks is not None:
        # Options (attention sinks) go through the _ex entry points.
        _need_cuda(sinks)
        if sinks.dtype != torch.float32 or sinks.shape != (H,) or not sinks.is_contiguous():
            raise ValueError("sinks must be a contiguous float32 tensor of num_heads values")
        opts = AttnOpts(sinks.data_ptr(), ctypes.pointer(fp8) if fp8 is not None else None)
        entry = "pa_varlen_fwd_ex" if entry.startswith("pa_varlen") else "pa_cascade_fwd_ex"
        if fp8 is not None:
            args = args[:20] + args[21:]          # the descriptor travels in opts
        code = getattr(lib, entry)(upd, *args[:20], ctypes.byref(opts), *args[20:])
        _check(code, entry)
        return out, lse
    fn = getattr(lib, entry)
    code = fn(upd, *args) if entry.endswith(("_with_update", "_fp8kv")) else fn(*args)
    _check(code, entry)
    return out, lse


def varlen_fwd(q, key_cache, value_cache, cu_seqlens_q, seqused_k, block_table, max_seqlen_q,
               max_seqlen_k, softmax_scale, causal, out=None, lse=None, return_lse=True,
               workspace=None, dev_status=None, sinks=None):
    """Varlen attention over a paged KV cache. Returns (out, lse or None)."""
    return _attend("pa_varlen_fwd", None, q, key_cache, value_cache, cu_seqlens_q, seqused_k,
                   block_table, max_seqlen_q, max_seqlen_k, softmax_scale, bool(causal), out,
                   lse, return_lse, workspace, dev_status, varlen_fwd_workspace_size, sinks=sinks)


def varlen_fwd_with_update(key, value, slot_mapping, q, key_cache, value_cache, cu_seqlens_q,
                           seqused_k, block_table, max_seqlen_q, max_seqlen_k, softmax_scale,
                           causal, out=None, lse=None, return_lse=True, workspace=None,
                           dev_status=None, sinks=None):
    """One step: scatter the new tokens' K/V (key, value by slot_mapping) into
    the caches, then varlen attention; the planner overlaps the scatter.
    Returns (out, lse or None)."""
    return _attend("pa_varlen_fwd_with_update", _kv_update(key, value, slot_mapping), q,
                   key_cache, value_cache, cu_seqlens_q, seqused_k, block_table, max_seqlen_q,
                   max_seqlen_k, softmax_scale, bool(causal), out, lse, return_lse, workspace,
                   dev_status, varlen_fwd_workspace_size, sinks=sinks,
                   update_tensors=(key, value))


def varlen_fwd_noalloc(q, key_cache, value_cache, cu_seqlens_q, seqused_k, block_table,
                       max_seqlen_q, max_seqlen_k, softmax_scale, causal, out=None, lse=None,
                       return_lse=True, dev_status=None):
    """varlen_fwd without a workspace: the library's fixed 32 MiB scratch is
    used instead (for callers that cannot allocate device memory). Calls that
    overlap on the GPU race on that buffer. Returns (out, lse or None)."""
    lib = load_library()
    _attn_common(q, key_cache, value_cache, cu_seqlens_q, seqused_k, block_table)
    T, H, D = q.shape
    nb, bs, hk, _ = key_cache.shape
    S = cu_seqlens_q.numel() - 1
    if out is None:
        out = torch.empty((T, H, D), dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    code = lib.pa_varlen_fwd_noalloc(
        _ptr(q), _row_stride(q), _ptr(key_cache), _ptr(value_cache), _cache_stride(key_cache),
        _ptr(cu_seqlens_q), _ptr(seqused_k), _ptr(block_table), block_table.stride(0), S, T,
        int(max_seqlen_q), int(max_seqlen_k), H, hk, D, bs, nb, float(softmax_scale),
        int(bool(causal)), _ptr(out), _ptr(lse), _dtype_code(q, out, key_cache, value_cache),
        _ptr(dev_status), _stream(q.device))
    _check(code, "pa_varlen_fwd_noalloc")
    return out, lse


def merge_attn_states(prefix_out, prefix_lse, suffix_out, suffix_lse, out=None, out_lse=None,
                      return_lse=True):
    """LSE-weighted combine of two partial attention states. Returns (out, lse or None)."""
    lib = load_library()
    _need_cuda(prefix_out, prefix_lse, suffix_out, suffix_lse)
    T, H, D = prefix_out.shape
    for t in (prefix_out, suffix_out):
        if not t.is_contiguous():
            raise ValueError("outputs must be contiguous [tokens, heads, head_size]")
    if out is None:
        out = torch.empty_like(prefix_out)
    if out_lse is None and return_lse:
        out_lse = torch.empty((H, T), dtype=torch.float32, device=prefix_out.device)
    code = lib.pa_merge_attn_states(
        _ptr(out), _ptr(out_lse), _ptr(prefix_out), _ptr(prefix_lse), _ptr(suffix_out),
        _ptr(suffix_lse), T, H, D, _dtype_code(prefix_out, suffix_out, out),
        _stream(prefix_out.device))
    _check(code, "pa_merge_attn_states")
    return out, out_lse


def merge_attn_states_n(parts_out, parts_lse, out=None, out_lse=None, return_lse=True):
    """LSE-weighted combine of n partial states: parts_out [n, T, H, D] bf16
    (each part contiguous), parts_lse [n, H, T] float32. Returns (out, lse or None)."""
    lib = load_library()
    _need_cuda(parts_out, parts_lse)
    n, T, H, D = parts_out.shape
    if parts_out[0].numel() and not parts_out[0].is_contiguous():
        raise ValueError("each part must be a contiguous [tokens, heads, head_size] tensor")
    if parts_lse.shape != (n, H, T) or (T and parts_lse.stride(2) != 1) or \
            (T and parts_lse.stride(1) != T):
        raise ValueError("parts_lse must be [n, heads, tokens] with contiguous parts")
    if out is None:
        out = torch.empty((T, H, D), dtype=parts_out.dtype, device=parts_out.device)
    if out_lse is None and return_lse:
        out_lse = torch.empty((H, T), dtype=torch.float32, device=parts_out.device)
    code = lib.pa_merge_attn_states_n(
        _ptr(out), _ptr(out_lse), _ptr(parts_out), parts_out.stride(0), _ptr(parts_lse),
        parts_lse.stride(0), n, T, H, D, _dtype_code(parts_out, out), _stream(parts_out.device))
    _check(code, "pa_merge_attn_states_n")
    return out, out_lse


def cascade_fwd(q, key_cache, value_cache, cu_seqlens_q, seqused_k, block_table, max_seqlen_q,
                max_seqlen_k, softmax_scale, common_prefix_len, out=None, lse=None,
                return_lse=True, workspace=None, dev_status=None, sinks=None):
    """Shared-prefix (cascade) attention. Returns (out, lse or None)."""
    return _attend("pa_cascade_fwd", None, q, key_cache, value_cache, cu_seqlens_q, seqused_k,
                   block_table, max_seqlen_q, max_seqlen_k, softmax_scale, common_prefix_len,
                   out, lse, return_lse, workspace, dev_status, cascade_fwd_workspace_size, sinks=sinks)


def cascade_fwd_with_update(key, value, slot_mapping, q, key_cache, value_cache, cu_seqlens_q,
                            seqused_k, block_table, max_seqlen_q, max_seqlen_k, softmax_scale,
                            common_prefix_len, out=None, lse=None, return_lse=True,
                            workspace=None, dev_status=None, sinks=None):
    """One step: scatter the new tokens' K/V into the caches, then cascade
    attention. Returns (out, lse or None)."""
    return _attend("pa_cascade_fwd_with_update", _kv_update(key, value, slot_mapping), q,
                   key_cache, value_cache, cu_seqlens_q, seqused_k, block_table, max_seqlen_q,
                   max_seqlen_k, softmax_scale, common_prefix_len, out, lse, return_lse,
                   workspace, dev_status, cascade_fwd_workspace_size, sinks=sinks,
                   update_tensors=(key, value))


# ---------------------------------------------------------------------------
# FP8 (e4m3) KV cache: uint8 (or float8_e4m3fn) pools of e4m3 codes with one
# scale per KV head; a stored code c means e4m3(c) * scale.
def _fp8_pool(c):
    if c.element_size() != 1:
        raise ValueError("FP8 caches hold one byte per element (uint8 or float8_e4m3fn)")
    return c


def _scales(s, hk, device):
    """Per-KV-head float32 scales on the device: a number, or a tensor of 1 or
    num_kv_heads values."""
    if not torch.is_tensor(s):
        return torch.full((hk,), float(s), dtype=torch.float32, device=device)
    if s.dtype == torch.float32 and s.shape == (hk,) and s.device == device and s.is_contiguous():
        return s
    s = s.to(device=device, dtype=torch.float32).reshape(-1)
    if s.numel() == 1:
        s = s.expand(hk)
    if s.numel() != hk:
        raise ValueError(f"expected 1 or {hk} scales, got {s.numel()}")
    return s.contiguous()


def _fp8_desc(k_scale, v_scale, hk, device):
    ks, vs = _scales(k_scale, hk, device), _scales(v_scale, hk, device)
    return KvFp8(ks.data_ptr(), vs.data_ptr()), (ks, vs)


def varlen_fwd_fp8kv_workspace_size(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads,
                                    num_kv_heads, head_size, block_size, sm_count):
    return load_library().pa_varlen_fwd_fp8kv_workspace_size(
        num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_size,
        block_size, sm_count)


def cascade_fwd_fp8kv_workspace_size(num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads,
                                     num_kv_heads, head_size, block_size, sm_count):
    return load_library().pa_cascade_fwd_fp8kv_workspace_size(
        num_seqs, total_q, max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_size,
        block_size, sm_count)


def reshape_and_cache_fp8(key, value, key_cache, value_cache, slot_mapping, k_scale, v_scale,
                          dev_status=None):
    """Quantize new bf16 K/V rows to e4m3 (x / scale of their KV head) and
    scatter them into the FP8 pools (in place)."""
    lib = load_library()
    _need_cuda(key, value, key_cache, value_cache, slot_mapping, dev_status)
    _fp8_pool(key_cache), _fp8_pool(value_cache)
    if key_cache.stride(0) != value_cache.stride(0):
        raise ValueError("key and value caches must share the page stride")
    nb, bs, hk, d = key_cache.shape
    desc, keep = _fp8_desc(k_scale, v_scale, hk, key.device)
    code = lib.pa_reshape_and_cache_fp8(
        _ptr(key), _ptr(value), _row_stride(key), _row_stride(value), _ptr(key_cache),
        _ptr(value_cache), _cache_stride(key_cache), _ptr(slot_mapping), key.shape[0], hk, d, bs,
        nb, ctypes.byref(desc), _dtype_code(key, value), _ptr(dev_status), _stream(key.device))
    _check(code, "pa_reshape_and_cache_fp8")
    del keep


def varlen_fwd_fp8kv(q, key_cache, value_cache, cu_seqlens_q, seqused_k, block_table,
                     max_seqlen_q, max_seqlen_k, softmax_scale, causal, k_scale, v_scale,
                     key=None, value=None, slot_mapping=None, out=None, lse=None,
                     return_lse=True, workspace=None, dev_status=None, sinks=None):
    """Varlen attention over FP8 pools, optionally first quantizing and
    scattering the new tokens' K/V (key, value, slot_mapping). Returns
    (out, lse or None)."""
    _fp8_pool(key_cache), _fp8_pool(value_cache)
    desc, keep = _fp8_desc(k_scale, v_scale, key_cache.shape[2], q.device)
    res = _attend("pa_varlen_fwd_fp8kv", _kv_update(key, value, slot_mapping), q, key_cache,
                  value_cache, cu_seqlens_q, seqused_k, block_table, max_seqlen_q, max_seqlen_k,
                  softmax_scale, bool(causal), out, lse, return_lse, workspace, dev_status,
                  varlen_fwd_fp8kv_workspace_size, fp8=desc, sinks=sinks,
                  update_tensors=(key, value))
    del keep
    return res


def cascade_fwd_fp8kv(q, key_cache, value_cache, cu_seqlens_q, seqused_k, block_table,
                      max_seqlen_q, max_seqlen_k, softmax_scale, common_prefix_len, k_scale,
                      v_scale, key=None, value=None, slot_mapping=None, out=None, lse=None,
                      return_lse=True, workspace=None, dev_status=None, sinks=None):
    """Cascade attention over FP8 pools (optional update as in
    varlen_fwd_fp8kv). Returns (out, lse or None)."""
    _fp8_pool(key_cache), _fp8_pool(value_cache)
    desc, keep = _fp8_desc(k_scale, v_scale, key_cache.shape[2], q.device)
    res = _attend("pa_cascade_fwd_fp8kv", _kv_update(key, value, slot_mapping), q, key_cache,
                  value_cache, cu_seqlens_q, seqused_k, block_table, max_seqlen_q, max_seqlen_k,
                  softmax_scale, common_prefix_len, out, lse, return_lse, workspace, dev_status,
                  cascade_fwd_fp8kv_workspace_size, fp8=desc, sinks=sinks,
                  update_tensors=(key, value))
    del keep
    return res


# ---------------------------------------------------------------------------
# Sliding window with first tokens
def _cu_seqlens(cu):
    """Number of sequences of cu_seqlens_q."""
    shape = cu.shape
    if cu.dtype is not torch.int32 or len(shape) != 1 or shape[0] < 1 or not cu.is_contiguous():
        raise ValueError("cu_seqlens_q must be a contiguous int32 tensor of num_seqs + 1 values")
    return shape[0] - 1


def window_fwd(q, key_cache, value_cache, cu_seqlens_q, seqused_k, block_table, max_seqlen_q,
               max_seqlen_k, softmax_scale, window, num_first=0, sinks=None, k_scale=None,
               v_scale=None, key=None, value=None, slot_mapping=None, out=None, lse=None,
               return_lse=True, workspace=None, dev_status=None):
    """Causal varlen attention in which a query sees its last window keys (its
    own among them) and the first num_first keys of its sequence; optionally
    the new tokens' K/V are first scattered into the caches (key, value,
    slot_mapping). With k_scale and v_scale the caches hold e4m3 bytes.
    Returns (out, lse or None)."""
    lib = load_library()
    mq, mk, window, first = int(max_seqlen_q), int(max_seqlen_k), int(window), int(num_first)
    if (mq | mk | window | first) >> 31:
        window, first = min(window, _INT_MAX), min(first, _INT_MAX)
        _fit32(mq, mk, window, first)
    if (key is None) is not (value is None) or (key is None) is not (slot_mapping is None):
        raise ValueError("key, value and slot_mapping go together")
    _one_device(q, key_cache, value_cache, cu_seqlens_q, seqused_k, block_table, sinks, key, value,
                slot_mapping, out, lse, workspace, dev_status)
    (nb, bs, hk, d), page = _pools(key_cache, value_cache)
    T, H, D = q.shape
    S = _cu_seqlens(cu_seqlens_q)
    bt_row = _seq_table(seqused_k, block_table, S)
    if d != D:
        raise ValueError("q and the caches must share the head size")
    if (k_scale is None) != (v_scale is None):
        raise ValueError("k_scale and v_scale go together")
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else q.new_empty((T, H, D))
    elif out.shape != (T, H, D) or not out.is_contiguous():
        raise ValueError("out must be a contiguous [total_q, num_heads, head_size] tensor")
    if lse is None:
        if return_lse:
            lse = q.new_empty((H, T), dtype=torch.float32)
    elif lse.dtype != torch.float32 or lse.shape != (H, T) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [num_heads, total_q] tensor")
    _f32_vector(sinks, H, "sinks")
    new, update = (), None
    if key is not None:
        new = (key, value)
        n = key.shape[0]
        if key.shape != (n, hk, D) or value.shape != (n, hk, D):
            raise ValueError("key and value must be [tokens, num_kv_heads, head_size]")
        if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (n,) or \
                not slot_mapping.is_contiguous():
            raise ValueError("slot_mapping must be a contiguous int64 tensor of one value per "
                             "token")
        update = KvUpdate(key.data_ptr(), value.data_ptr(), _row_stride(key), _row_stride(value),
                          slot_mapping.data_ptr(), n)
    desc = keep = None
    if k_scale is None:
        dtype = _dtype_code(q, out, key_cache, value_cache, *new)
    else:
        _fp8_pool(key_cache), _fp8_pool(value_cache)
        dtype = _dtype_code(q, out, *new)
        desc, keep = _fp8_desc(k_scale, v_scale, hk, q.device)
    if workspace is None:
        size = varlen_fwd_workspace_size if desc is None else varlen_fwd_fp8kv_workspace_size
        workspace = alloc_workspace(size(S, T, mq, mk, H, hk, D, bs, _sm_count(q.device)),
                                    q.device)
    opts = None
    if sinks is not None or desc is not None:
        opts = ctypes.byref(AttnOpts(_ptr(sinks), None if desc is None else ctypes.pointer(desc)))
    _call(lib.pa_window_fwd, "pa_window_fwd", q.device,
          None if update is None else ctypes.byref(update), q.data_ptr(), _row_stride(q),
          key_cache.data_ptr(), value_cache.data_ptr(), page, cu_seqlens_q.data_ptr(),
          seqused_k.data_ptr(), block_table.data_ptr(), bt_row, S, T, mq, mk, H, hk, D, bs, nb,
          float(softmax_scale), window, first, opts, out.data_ptr(), _ptr(lse),
          workspace.data_ptr(), workspace.numel(), dtype, _ptr(dev_status))
    del keep
    return out, lse


# ---------------------------------------------------------------------------
# Rotary positions
def rope_table(table_len, rot_dim, base=10000.0, scaling="none", factor=1.0, orig_len=0.0,
               low=None, high=None, mscale=None, out=None, device="cuda"):
    """Rotary cos/sin table float32 [table_len, rot_dim] (row: rot_dim / 2
    cosines, then sines). scaling: "none", "linear", "ntk", "wavelength" (low,
    high turns within orig_len, default 1 and 4) or "yarn" (default 1 and 32;
    mscale default 0.1 ln factor + 1 for factor > 1)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    _fit32(table_len, rot_dim)
    if out is None:
        out = torch.empty((table_len, rot_dim), dtype=torch.float32, device=device)
    _need_cuda(out)
    if out.dtype != torch.float32 or out.shape != (table_len, rot_dim) or not out.is_contiguous():
        raise ValueError("out must be a contiguous float32 [table_len, rot_dim] tensor")
    if mscale is None:
        mscale = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1 else 1.0
    desc = RopeScaling(ROPE_SCALINGS[scaling], factor, orig_len, 1.0 if low is None else low,
                       (32.0 if scaling == "yarn" else 4.0) if high is None else high, mscale)
    _call(load_library().pa_rope_table, "pa_rope_table", out.device, _ptr(out), int(table_len),
          int(rot_dim), float(base), ctypes.byref(desc))
    return out


def _f32_vector(t, n, name):
    if t is not None and (t.dtype != torch.float32 or t.shape != (n,) or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous float32 tensor of {n} values")


def rope_and_cache(q, key, value, positions, cos_sin, key_cache, value_cache, slot_mapping,
                   interleaved=False, q_norm=None, k_norm=None, eps=1e-6, k_scale=None,
                   v_scale=None, out=None, dev_status=None):
    """Norm (optional weights q_norm, k_norm) and rotate the new queries and
    keys by the table rows of their positions, and write keys and values into
    their pages (in place on the caches; with k_scale and v_scale the caches
    hold e4m3 bytes). Returns the rotated queries; out may be q itself."""
    lib = load_library()
    rows, rot = cos_sin.shape
    if rows >> 31:
        _fit32(rows)
    _one_device(q, key, value, positions, cos_sin, key_cache, value_cache, slot_mapping, q_norm,
                k_norm, out, dev_status)
    (nb, bs, hk, d), page = _pools(key_cache, value_cache)
    T, H, dq = q.shape
    row = (T, hk, d)
    if dq != d or key.shape != row or value.shape != row:
        raise ValueError("q, key and value must be [tokens, heads, head_size] of the caches' "
                         "heads and head size")
    if positions.dtype is not torch.int64 or positions.shape != (T,) or \
            not positions.is_contiguous() or slot_mapping.dtype is not torch.int64 or \
            slot_mapping.shape != (T,) or not slot_mapping.is_contiguous():
        raise ValueError("positions and slot_mapping must be contiguous int64 tensors of one "
                         "value per token")
    if cos_sin.dtype != torch.float32 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be a contiguous float32 [positions, rot_dim] tensor")
    _f32_vector(q_norm, d, "q_norm")
    _f32_vector(k_norm, d, "k_norm")
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else q.new_empty((T, H, d))
        out_row = H * d
    elif out.shape != q.shape:
        raise ValueError("out must have the shape of q")
    else:
        out_row = _row_stride(out)
    if k_scale is None and v_scale is None:
        dtype, fp8, keep = _dtype_code(q, key, value, out, key_cache, value_cache), None, None
    elif k_scale is None or v_scale is None:
        raise ValueError("k_scale and v_scale go together")
    else:
        _fp8_pool(key_cache), _fp8_pool(value_cache)
        dtype = _dtype_code(q, key, value, out)
        desc, keep = _fp8_desc(k_scale, v_scale, hk, q.device)
        fp8 = ctypes.byref(desc)
    rope = Rope(cos_sin.data_ptr(), rows, rot, 1 if interleaved else 0, _ptr(q_norm),
                _ptr(k_norm), eps)
    update = KvUpdate(key.data_ptr(), value.data_ptr(), _row_stride(key), _row_stride(value),
                      slot_mapping.data_ptr(), T)
    _call(lib.pa_rope_and_cache, "pa_rope_and_cache", q.device,
          ctypes.byref(rope), positions.data_ptr(), q.data_ptr(), _row_stride(q), out.data_ptr(),
          out_row, ctypes.byref(update), key_cache.data_ptr(), value_cache.data_ptr(),
          page, H, hk, d, bs, nb, fp8, dtype, _ptr(dev_status))
    del keep
    return out


# ---------------------------------------------------------------------------
# Accumulated attention weight of the cached keys, and eviction by it
def _weights_stride(weights, nb, bs, hk):
    """Page stride of a weights tensor [num_blocks, num_kv_heads, block_size]."""
    st = weights.stride()
    if weights.dtype is not torch.float32 or weights.shape != (nb, hk, bs) or st[2] != 1 or \
            st[1] != bs:
        raise ValueError("weights must be float32 [num_blocks, num_kv_heads, block_size] with "
                         "contiguous pages")
    return st[0]


def attn_weights(q, key_cache, lse, weights, cu_seqlens_q, seqused_k, block_table, max_seqlen_q,
                 max_seqlen_k, softmax_scale, causal, k_scale=None, dev_status=None):
    """Add the attention weight that this call's queries gave every cached key
    (recomputed from K and the attention call's lse) to weights, float32
    [num_blocks, num_kv_heads, block_size], in place; the keys of the call's
    own queries start from zero. With k_scale the key cache holds e4m3 bytes.
    A sequence's pages must be its own: a page that two sequences of the call
    share (a common prefix) gets the sum of one of them. Returns weights."""
    lib = load_library()
    mq, mk = int(max_seqlen_q), int(max_seqlen_k)
    if (mq | mk) >> 31:
        _fit32(mq, mk)
    _one_device(q, key_cache, lse, weights, cu_seqlens_q, seqused_k, block_table, dev_status)
    S = _cu_seqlens(cu_seqlens_q)
    bt_row = _seq_table(seqused_k, block_table, S)
    T, H, D = q.shape
    nb, bs, hk, d = key_cache.shape
    if d != D:
        raise ValueError("q and the key cache must share the head size")
    if lse.dtype != torch.float32 or lse.shape != (H, T) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [num_heads, total_q] tensor")
    desc = keep = None
    if k_scale is not None:
        _fp8_pool(key_cache)
        desc, keep = _fp8_desc(k_scale, k_scale, hk, q.device)
    dtype = _dtype_code(q) if desc is not None else _dtype_code(q, key_cache)
    _call(lib.pa_attn_weights, "pa_attn_weights", q.device,
          _ptr(q), _row_stride(q), _ptr(key_cache), _cache_stride(key_cache), _ptr(lse),
          _ptr(cu_seqlens_q), _ptr(seqused_k), _ptr(block_table), bt_row,
          S, T, mq, mk, H, hk, D, bs, nb, float(softmax_scale), int(bool(causal)), _ptr(weights),
          _weights_stride(weights, nb, bs, hk), None if desc is None else ctypes.byref(desc),
          dtype, _ptr(dev_status))
    del keep
    return weights


def evict(key_cache, value_cache, weights, seqused_k, block_table, max_seqlen_k, budget,
          num_first=0, num_recent=0, kept=None, new_lens=None, dev_status=None):
    """Cut every sequence of more than budget keys down to budget, per KV head:
    its first num_first keys, its last num_recent and the heaviest of the rest
    by weights; kept rows of the caches (2-byte or e4m3 elements) and of
    weights move to the front of the sequence's pages, which must be its own
    (none shared with another sequence: rows are rewritten in place). Returns
    (kept int32 [num_seqs, num_kv_heads, budget], new_lens int32 [num_seqs]);
    new_lens may be seqused_k itself."""
    lib = load_library()
    mk, budget, first, recent = int(max_seqlen_k), int(budget), int(num_first), int(num_recent)
    if (mk | budget | first | recent) >> 31:
        _fit32(mk, budget, first, recent)
    _one_device(key_cache, value_cache, weights, seqused_k, block_table, kept, new_lens,
                dev_status)
    (nb, bs, hk, d), page = _pools(key_cache, value_cache)
    if key_cache.dtype is not value_cache.dtype:
        raise ValueError("key and value caches must have the same type")
    S = seqused_k.numel()
    row = _seq_table(seqused_k, block_table, S)
    device = key_cache.device
    if kept is None:
        kept = seqused_k.new_empty((S, hk, max(budget, 0)))
    elif kept.dtype != torch.int32 or kept.shape != (S, hk, budget) or not kept.is_contiguous():
        raise ValueError("kept must be a contiguous int32 [num_seqs, num_kv_heads, budget] tensor")
    if new_lens is None:
        new_lens = torch.empty_like(seqused_k)
    elif new_lens.dtype != torch.int32 or new_lens.shape != (S,) or not new_lens.is_contiguous():
        raise ValueError("new_lens must be a contiguous int32 tensor of one value per sequence")
    _call(lib.pa_evict, "pa_evict", device,
          key_cache.data_ptr(), value_cache.data_ptr(), page, weights.data_ptr(),
          _weights_stride(weights, nb, bs, hk), seqused_k.data_ptr(), block_table.data_ptr(),
          row, S, mk, hk, d, bs, nb, key_cache.element_size(), budget, first, recent,
          kept.data_ptr(), new_lens.data_ptr(), _ptr(dev_status))
    return kept, new_lens
