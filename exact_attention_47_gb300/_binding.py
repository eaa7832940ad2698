"""ctypes binding of ``libattn47_sm103.so`` (argument marshalling only).

Every function here checks tensor properties the C-ABI cannot see (device,
dtype, contiguity, shapes), allocates outputs with torch when the caller
passes none, and forwards raw device pointers plus the current torch CUDA
stream to the C entry point of the same name.  All arithmetic runs in the
library's CUDA kernels; there is no other code path.  If the library is not
built, every call raises ``RuntimeError``.
"""

import ctypes
import functools
import importlib.machinery
import importlib.util
import os
import struct
import warnings

import torch

from .build_lib import LIB_PATH, fast_path

ATTN_OK = 0
ATTN_DEV_TIMEOUT = 0x1
ATTN_DEV_BAD_BLOCK = 0x2
ATTN_DEV_BAD_SEQLEN = 0x4
ATTN_DEV_BAD_SEQID = 0x8
BLOCK_SIZE = 16

# C entry points and their signatures (mirrors include/attn47.h)
_P = ctypes.c_void_p
_I = ctypes.c_int
_SIGS = {
    "attn_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P]),
    "attn_bwd_workspace_size": (ctypes.c_size_t, [_I, _I, _I]),
    "attn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float,
                      _P, ctypes.c_size_t, _P]),
    "attn_decode_paged_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "attn_decode_paged": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float,
                               _P, _P, _P, ctypes.c_size_t, _P]),
    "attn_decode_paged_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float,
                                       _P, _P, _P]),
    "attn_prefill_paged": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I,
                                ctypes.c_float, _P, _P, _P]),
    "fused_add_rmsnorm": (_I, [_P, _P, _P, _P, _I, _I, ctypes.c_float, _P]),
    "fused_swiglu": (_I, [_P, _P, _I, _I, _P]),
    "swiglu_projection": (_I, [_P, _P, _P, _I, _I, _I, _P]),
    "ssd_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I, _I]),
    "ssd_chunked_fwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P,
                             ctypes.c_size_t, _P]),
    "rope_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "rope_bwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "rope_append_paged": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "kv4_record_bytes": (ctypes.c_size_t, [_I, _I]),
    "rope_append_paged_kv4": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "kv8_record_bytes": (ctypes.c_size_t, [_I]),
    "kv8_append_paged": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "kv8_read_paged": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P]),
    "attn_decode_paged_kv8_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "attn_decode_paged_kv8": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P,
                                   ctypes.c_size_t, _P]),
    "attn_prefill_paged_kv8_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I, _I]),
    "attn_prefill_paged_kv8": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P,
                                    ctypes.c_size_t, _P]),
    "kv4_read_paged": (_I, [_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P]),
    "attn_decode_paged_kv4_workspace_size": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "attn_decode_paged_kv4": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P,
                                   ctypes.c_size_t, _P]),
    "attn_get_device_status": (_I, [_P, ctypes.POINTER(ctypes.c_uint)]),
    "attn_set_wait_timeout_ns": (None, [ctypes.c_ulonglong]),
    "attn_set_decode_max_ctas": (None, [_I]),
    "attn_set_decode_early_plan": (None, [_I]),
    "attn_selftest_wait_timeout": (_I, [ctypes.c_ulonglong, _P, ctypes.POINTER(ctypes.c_uint)]),
    "attn_selftest_exp2_poly": (_I, [_P, _P, _I, _P]),
    "attn_status_string": (ctypes.c_char_p, [_I]),
    "attn_last_error": (ctypes.c_char_p, []),
    "attn_abi_version": (_I, []),
}



# attn_heads_t and attn_rope_t of include/attn47.h, packed as bytes (their
# address goes to the library): a ctypes structure costs several times as much
# to fill, and a decode step's small calls are bound by the host.
_HEADS = struct.Struct("Pqqqi")
_ROPE = struct.Struct("PiiPiqqP")


_lib = None


class AttnError(RuntimeError):
    """A non-zero attn_status_t from the library."""

    def __init__(self, func, status, message):
        self.status = status
        super().__init__("%s failed: %s: %s" % (func, status_string(status), message))


def library_path():
    return LIB_PATH


def load_library(path=None):
    """Load (once) and return the ctypes handle of the CUDA library."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(
            "CUDA library %s is not built; run `python -c \"import __graft_entry__ as g; g.build()\"` "
            "(there is no CPU fallback)" % path)
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


# The entry points that the fast calls pass on to, in the order of their `bind`.
_FAST = ("rope_fwd", "rope_bwd", "rope_append_paged", "rope_append_paged_kv4", "kv4_record_bytes", "kv4_read_paged",
         "attn_decode_paged_kv4_workspace_size", "attn_decode_paged_kv4")
# Those of the 8-bit cache, in the order of `bind8`.
_FAST_KV8 = ("kv8_append_paged", "kv8_record_bytes", "kv8_read_paged", "attn_decode_paged_kv8_workspace_size",
             "attn_decode_paged_kv8", "attn_prefill_paged_kv8_workspace_size", "attn_prefill_paged_kv8")


class _NoFastCalls:
    """In place of the module of the fast calls where it is not built: nothing
    is the usual case, every call goes the Python way."""

    @staticmethod
    def rope(*args):
        return None

    append = read = decode = append8 = read8 = decode8 = prefill8 = rope


@functools.lru_cache(maxsize=None)
def _fast():
    """The module of the fast calls (csrc/fast_calls.cpp), bound to the
    library.  Each takes the arguments of its namesake here, and does the call
    or returns None where it is not the usual case, or the status of a call that
    was made and failed."""
    lib = load_library()
    path = fast_path()
    if not os.path.exists(path):
        warnings.warn("%s is not built (it takes g++ and the headers of Python and torch): the rotary, append, "
                      "8- and 4-bit-cache calls cost more host time" % path, RuntimeWarning, stacklevel=3)
        return _NoFastCalls
    loader = importlib.machinery.ExtensionFileLoader("_attn47_fast", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_attn47_fast", loader))
    loader.exec_module(module)
    module.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _FAST))
    module.bind8(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _FAST_KV8))
    return module


def status_string(status):
    return load_library().attn_status_string(int(status)).decode()


def _check(func, status):
    if status != ATTN_OK:
        raise AttnError(func, status, load_library().attn_last_error().decode())


def _stream_handle(stream, device=None):
    """The raw cudaStream_t of `stream` (default: torch's current stream of
    `device`); a stream of another device is refused."""
    if stream is None:
        if device is not None and device.index is not None:
            return torch._C._cuda_getCurrentRawStream(device.index)   # no Stream object made
        stream = torch.cuda.current_stream(device)
    elif device is not None and stream.device != device:
        raise ValueError("stream is on %s but the tensors are on %s" % (stream.device, device))
    return stream.cuda_stream


def _on_stream(func, stream, tensor, *args):
    """func(*args) with `stream` current, which is then also the one that what
    the call allocates belongs to."""
    if isinstance(tensor, torch.Tensor) and tensor.is_cuda:
        _stream_handle(stream, tensor.device)
    with torch.cuda.stream(stream):
        return func(*args)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _need_cuda(name, t, dtype, device=None, contiguous=True):
    """`t` is a (contiguous) CUDA tensor of `dtype` (any dtype if None) on
    `device` (if given)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if (t.is_cuda and (dtype is None or t.dtype is dtype) and (device is None or t.device == device)
            and (not contiguous or t.is_contiguous())):
        return
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, the other tensors on %s" % (name, t.device, device))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _need_shape(name, t, shape):
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _output(name, t, shape, dtype, device):
    """A caller-given output checked for device, dtype and shape, or a new one."""
    if t is None:
        return torch.empty(tuple(shape), dtype=dtype, device=device)
    _need_cuda(name, t, dtype, device)
    _need_shape(name, t, shape)
    return t


def _workspace(name, t, need, device):
    """A caller-given workspace (any dtype, contiguous, on `device`, at least
    `need` bytes), or a new one of `need` bytes."""
    if t is None:
        return torch.empty(max(int(need), 16), dtype=torch.uint8, device=device)
    _need_cuda(name, t, None, device)
    nbytes = t.numel() * t.element_size()
    if nbytes < need:
        raise ValueError("%s has %d bytes, needs %d" % (name, nbytes, need))
    return t


def _call(func, device, *args):
    """Call C entry point `func` with `device` current and raise on error."""
    fn = getattr(load_library(), func)
    if torch.cuda.current_device() == device.index:
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    if st != ATTN_OK:
        _check(func, st)


def attn_fwd(q, k, v, causal=True, scale=None, o=None, lse=None, return_lse=True, stream=None):
    """Exact attention forward.  q [B,Hq,N,d], k/v [B,Hkv,N,d] bf16 on the GPU.

    Returns (o, lse): o [B,Hq,N,d] bf16, lse [B,Hq,N] fp32 (None when
    ``return_lse`` is False and no ``lse`` buffer is given).
    """
    _need_cuda("q", q, torch.bfloat16)
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need_cuda(name, t, torch.bfloat16, dev)
        if t.dim() != 4:
            raise ValueError("%s must be 4-D [B, H, N, d]" % name)
    B, Hq, N, d = q.shape
    if k.shape[0] != B or k.shape[2] != N or k.shape[3] != d or v.shape != k.shape:
        raise ValueError("k and v must be [B, Hkv, N, d] matching q")
    Hkv = k.shape[1]
    if scale is None:
        scale = d ** -0.5
    o = _output("o", o, q.shape, torch.bfloat16, dev)
    if lse is not None or return_lse:
        lse = _output("lse", lse, (B, Hq, N), torch.float32, dev)
    _call("attn_fwd", dev, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d,
          1 if causal else 0, float(scale), _stream_handle(stream, dev))
    return o, lse


def attn_bwd_workspace_size(B, Hq, N):
    return int(load_library().attn_bwd_workspace_size(B, Hq, N))


def attn_bwd(q, k, v, o, lse, dout, causal=True, scale=None, dq=None, dk=None, dv=None,
             workspace=None, stream=None):
    """Gradients of attn_fwd.  q/o/dout [B,Hq,N,d], k/v [B,Hkv,N,d] bf16 and
    lse [B,Hq,N] fp32 (attn_fwd's outputs for the same inputs), on the GPU.

    Returns (dq [B,Hq,N,d], dk [B,Hkv,N,d], dv [B,Hkv,N,d]) bf16.
    """
    _need_cuda("q", q, torch.bfloat16)
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _need_cuda(name, t, torch.bfloat16, dev)
        if t.dim() != 4:
            raise ValueError("%s must be 4-D [B, H, N, d]" % name)
    _need_cuda("lse", lse, torch.float32, dev)
    B, Hq, N, d = q.shape
    if k.shape[0] != B or k.shape[2] != N or k.shape[3] != d or v.shape != k.shape:
        raise ValueError("k and v must be [B, Hkv, N, d] matching q")
    _need_shape("o", o, q.shape)
    _need_shape("dout", dout, q.shape)
    _need_shape("lse", lse, (B, Hq, N))
    Hkv = k.shape[1]
    if scale is None:
        scale = d ** -0.5
    dq = _output("dq", dq, q.shape, torch.bfloat16, dev)
    dk = _output("dk", dk, k.shape, torch.bfloat16, dev)
    dv = _output("dv", dv, v.shape, torch.bfloat16, dev)
    workspace = _workspace("workspace", workspace, attn_bwd_workspace_size(B, Hq, N), dev)
    _call("attn_bwd", dev, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq),
          _ptr(dk), _ptr(dv), B, Hq, Hkv, N, d, 1 if causal else 0, float(scale), _ptr(workspace),
          workspace.numel() * workspace.element_size(), _stream_handle(stream, dev))
    return dq, dk, dv


def attn_decode_paged_workspace_size(num_seqs, Hq, d, max_blocks_per_seq):
    return int(load_library().attn_decode_paged_workspace_size(num_seqs, Hq, d, max_blocks_per_seq))


def _decode_args(q, k_cache, v_cache, block_table, seq_lens, scale, o, lse, return_lse):
    """Checks shared by both decode entry points; returns the sizes, the
    scale and the (checked or new) outputs."""
    _need_cuda("q", q, torch.bfloat16)
    dev = q.device
    for name, t, dt in (("k_cache", k_cache, torch.bfloat16), ("v_cache", v_cache, torch.bfloat16),
                        ("block_table", block_table, torch.int32), ("seq_lens", seq_lens, torch.int32)):
        _need_cuda(name, t, dt, dev)
    if q.dim() != 3 or k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("q must be [S,Hq,d] and caches [num_blocks,Hkv,block_size,d]")
    S, Hq, d = q.shape
    num_blocks, Hkv, block_size, dc = k_cache.shape
    if dc != d:
        raise ValueError("cache head dim %d differs from q's %d" % (dc, d))
    if block_table.dim() != 2 or block_table.shape[0] != S:
        raise ValueError("block_table must be [S, max_blocks]")
    _need_shape("seq_lens", seq_lens, (S,))
    o = _output("o", o, (S, Hq, d), torch.bfloat16, dev)
    if lse is not None or return_lse:
        lse = _output("lse", lse, (S, Hq), torch.float32, dev)
    if scale is None:
        scale = d ** -0.5
    return dev, S, Hq, Hkv, d, block_size, block_table.shape[1], num_blocks, float(scale), o, lse


def attn_decode_paged(q, k_cache, v_cache, block_table, seq_lens, scale=None, o=None, lse=None,
                      workspace=None, return_lse=True, stream=None):
    """Paged-KV decode.  q [S,Hq,d]; caches [num_blocks,Hkv,16,d] bf16;
    block_table [S,max_blocks] int32; seq_lens [S] int32 (all on the GPU).

    Returns (o [S,Hq,d] bf16, lse [S,Hq] fp32 or None).
    """
    dev, S, Hq, Hkv, d, bs, mb, nb, scale, o, lse = _decode_args(
        q, k_cache, v_cache, block_table, seq_lens, scale, o, lse, return_lse)
    workspace = _workspace("workspace", workspace, attn_decode_paged_workspace_size(S, Hq, d, mb), dev)
    _call("attn_decode_paged", dev, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
          _ptr(seq_lens), S, Hq, Hkv, d, bs, mb, nb, scale, _ptr(o), _ptr(lse), _ptr(workspace),
          workspace.numel() * workspace.element_size(), _stream_handle(stream, dev))
    return o, lse


def attn_decode_paged_noalloc(q, k_cache, v_cache, block_table, seq_lens, scale=None, o=None,
                              lse=None, return_lse=True, stream=None):
    """attn_decode_paged without a workspace argument, for callers that may
    not allocate device memory when they run the decode: the library uses
    its own fixed 8 MiB device array instead (sizes needing more raise
    AttnError with ATTN_ERR_WORKSPACE).  Calls that overlap on the GPU share
    that array and must be ordered.  Only the outputs, if not given, are
    allocated here, by torch; pass ``o`` (and ``lse`` or return_lse=False)
    to allocate nothing at all."""
    dev, S, Hq, Hkv, d, bs, mb, nb, scale, o, lse = _decode_args(
        q, k_cache, v_cache, block_table, seq_lens, scale, o, lse, return_lse)
    _call("attn_decode_paged_noalloc", dev, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
          _ptr(seq_lens), S, Hq, Hkv, d, bs, mb, nb, scale, _ptr(o), _ptr(lse),
          _stream_handle(stream, dev))
    return o, lse


def attn_prefill_paged(q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, scale=None,
                       o=None, lse=None, return_lse=True, stream=None):
    """Chunked prefill over a paged cache (all tensors on the GPU).

    q [S,Hq,N,d], k_new / v_new [S,Hkv,N,d] bf16; caches
    [num_blocks,Hkv,16,d] bf16 (updated in place: the new rows are appended at
    positions ctx_lens[b] + i); block_table [S,max_blocks] int32; ctx_lens [S]
    int32 (left unchanged).  Returns (o [S,Hq,N,d] bf16, lse [S,Hq,N] fp32 or
    None).
    """
    _need_cuda("q", q, torch.bfloat16)
    dev = q.device
    for name, t, dt in (("k_new", k_new, torch.bfloat16), ("v_new", v_new, torch.bfloat16),
                        ("k_cache", k_cache, torch.bfloat16), ("v_cache", v_cache, torch.bfloat16),
                        ("block_table", block_table, torch.int32), ("ctx_lens", ctx_lens, torch.int32)):
        _need_cuda(name, t, dt, dev)
    if q.dim() != 4 or k_new.dim() != 4 or k_new.shape != v_new.shape:
        raise ValueError("q must be [S,Hq,N,d] and k_new / v_new [S,Hkv,N,d]")
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("caches must be [num_blocks,Hkv,block_size,d]")
    S, Hq, N, d = q.shape
    num_blocks, Hkv, block_size, dc = k_cache.shape
    if k_new.shape != (S, Hkv, N, d) or dc != d:
        raise ValueError("k_new / v_new must be [S, Hkv, N, d] matching q and the caches")
    if block_table.dim() != 2 or block_table.shape[0] != S:
        raise ValueError("block_table must be [S, max_blocks]")
    _need_shape("ctx_lens", ctx_lens, (S,))
    if scale is None:
        scale = d ** -0.5
    o = _output("o", o, q.shape, torch.bfloat16, dev)
    if lse is not None or return_lse:
        lse = _output("lse", lse, (S, Hq, N), torch.float32, dev)
    _call("attn_prefill_paged", dev, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
          _ptr(block_table), _ptr(ctx_lens), S, Hq, Hkv, N, d, block_size, block_table.shape[1],
          num_blocks, float(scale), _ptr(o), _ptr(lse), _stream_handle(stream, dev))
    return o, lse


def fused_add_rmsnorm(x, residual, weight, eps=1e-6, out=None, stream=None):
    """Residual add + RMSNorm.  x, residual [rows, hidden] and weight [hidden]
    bf16 on the GPU; ``residual`` is overwritten with bf16(x + residual).
    Returns (out [rows, hidden] bf16, residual)."""
    _need_cuda("x", x, torch.bfloat16)
    dev = x.device
    for name, t in (("residual", residual), ("weight", weight)):
        _need_cuda(name, t, torch.bfloat16, dev)
    if x.dim() != 2 or residual.shape != x.shape or weight.dim() != 1 or weight.shape[0] != x.shape[1]:
        raise ValueError("x and residual must be [rows, hidden] and weight [hidden]")
    rows, hidden = x.shape
    out = _output("out", out, x.shape, torch.bfloat16, dev)
    _call("fused_add_rmsnorm", dev, _ptr(x), _ptr(residual), _ptr(weight), _ptr(out), rows, hidden,
          float(eps), _stream_handle(stream, dev))
    return out, residual


def fused_swiglu(gate_up, out=None, stream=None):
    """SwiGLU activation of the merged gate/up projection output
    gate_up [rows, 2F] bf16 (gate first): returns silu(gate) * up [rows, F] bf16."""
    _need_cuda("gate_up", gate_up, torch.bfloat16)
    dev = gate_up.device
    if gate_up.dim() != 2 or gate_up.shape[1] % 2 != 0:
        raise ValueError("gate_up must be [rows, 2F]")
    rows, F = gate_up.shape[0], gate_up.shape[1] // 2
    out = _output("out", out, (rows, F), torch.bfloat16, dev)
    _call("fused_swiglu", dev, _ptr(gate_up), _ptr(out), rows, F, _stream_handle(stream, dev))
    return out


def swiglu_projection(x, w_gate_up, out=None, stream=None):
    """Gate/up projection with the SwiGLU activation fused in:
    x [rows, hidden] bf16, w_gate_up [2F, hidden] bf16 (gate rows first);
    returns silu(x W_gate^T) * (x W_up^T) [rows, F] bf16."""
    _need_cuda("x", x, torch.bfloat16)
    dev = x.device
    _need_cuda("w_gate_up", w_gate_up, torch.bfloat16, dev)
    if x.dim() != 2 or w_gate_up.dim() != 2 or w_gate_up.shape[1] != x.shape[1] or w_gate_up.shape[0] % 2:
        raise ValueError("x must be [rows, hidden] and w_gate_up [2F, hidden]")
    rows, hidden = x.shape
    F = w_gate_up.shape[0] // 2
    out = _output("out", out, (rows, F), torch.bfloat16, dev)
    _call("swiglu_projection", dev, _ptr(x), _ptr(w_gate_up), _ptr(out), rows, hidden, F,
          _stream_handle(stream, dev))
    return out


def ssd_workspace_size(batch, L, H, N, chunk):
    return int(load_library().ssd_workspace_size(batch, L, H, N, chunk))


def ssd_chunked_fwd(x, dt, A, B, C, chunk=256, h0=None, y=None, h_final=None, workspace=None,
                    stream=None):
    """Mamba-2 SSD forward.  x [batch, L, H, P] bf16, dt [batch, L, H] fp32,
    A [H] fp32, B and C [batch, L, G, N] bf16, h0 [batch, H, P, N] fp32 or
    None, all on the GPU.  Returns (y [batch, L, H, P] bf16, h_final
    [batch, H, P, N] fp32)."""
    _need_cuda("x", x, torch.bfloat16)
    dev = x.device
    for name, t, dtype in (("dt", dt, torch.float32), ("A", A, torch.float32),
                           ("B", B, torch.bfloat16), ("C", C, torch.bfloat16)):
        _need_cuda(name, t, dtype, dev)
    if x.dim() != 4 or dt.dim() != 3 or A.dim() != 1 or B.dim() != 4 or C.shape != B.shape:
        raise ValueError("x [batch, L, H, P], dt [batch, L, H], A [H], B/C [batch, L, G, N]")
    batch, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    if tuple(dt.shape) != (batch, L, H) or A.shape[0] != H or B.shape[:2] != x.shape[:2]:
        raise ValueError("dt, A, B and C do not match x")
    if h0 is not None:
        _need_cuda("h0", h0, torch.float32, dev)
        _need_shape("h0", h0, (batch, H, P, N))
    y = _output("y", y, x.shape, torch.bfloat16, dev)
    h_final = _output("h_final", h_final, (batch, H, P, N), torch.float32, dev)
    workspace = _workspace("workspace", workspace, ssd_workspace_size(batch, L, H, N, chunk), dev)
    _call("ssd_chunked_fwd", dev, _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(h0), _ptr(y),
          _ptr(h_final), batch, L, H, G, P, N, chunk, _ptr(workspace),
          workspace.numel() * workspace.element_size(), _stream_handle(stream, dev))
    return y, h_final


def _heads(name, t, device, dim):
    """attn_heads_t of a bf16 tensor [B, H, N, d] (``dim`` 4) or [T, H, d]
    (``dim`` 3), any strides but a contiguous last dimension."""
    _need_cuda(name, t, torch.bfloat16, device, contiguous=False)
    shape, stride = t.shape, t.stride()
    if len(shape) != dim:
        raise ValueError("%s must be %s" % (name, "[B, H, N, d]" if dim == 4 else "[T, H, d]"))
    if stride[-1] != 1 and shape[-1] > 1:
        raise ValueError("%s must have a contiguous last dimension" % name)
    # The stride of a dimension with one entry means nothing.
    if dim == 4:
        return _HEADS.pack(t.data_ptr(), stride[0] if shape[0] > 1 else 0, stride[2] if shape[2] > 1 else 0,
                           stride[1] if shape[1] > 1 else 0, shape[1])
    return _HEADS.pack(t.data_ptr(), 0, stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0, shape[1])


def _rope(inv_freq, positions, lead, pair_axis, interleaved, device):
    """attn_rope_t and what has to live as long as it.  ``lead`` is the shape
    that a position axis may have: (N,) or (B, N); ``positions`` is that, or
    with ``pair_axis`` [axes, ...that]."""
    _need_cuda("inv_freq", inv_freq, torch.float32, device)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [rot / 2]")
    pairs = inv_freq.shape[0]
    at, axes, stride_axis, stride_batch, table, table_at = 0, 1, 0, 0, None, 0
    if pair_axis is not None:
        if len(pair_axis) != pairs:
            raise ValueError("pair_axis has %d entries, inv_freq %d" % (len(pair_axis), pairs))
        if positions is None:
            raise ValueError("pair_axis needs positions with axes")
        table = ctypes.c_char_p(bytes(pair_axis))
        table_at = ctypes.cast(table, ctypes.c_void_p).value
    if positions is not None:
        _need_cuda("the rotation's positions", positions, torch.int32, device, contiguous=False)
        shape, stride = tuple(positions.shape), positions.stride()
        if pair_axis is not None:
            if not shape:
                raise ValueError("with pair_axis, positions must be [axes, ...]")
            axes, stride_axis = shape[0], stride[0] if shape[0] > 1 else 0
            shape, stride = shape[1:], stride[1:]
        if shape != lead and shape != lead[-1:]:
            raise ValueError("positions of an axis must have shape %s, got %s"
                             % (" or ".join(map(str, sorted({lead, lead[-1:]}))), shape))
        if len(shape) == 2 and shape[0] > 1:
            stride_batch = stride[0]
        if shape[-1] > 1 and stride[-1] != 1:
            raise ValueError("positions must have a contiguous last dimension")
        at = positions.data_ptr()
    return _ROPE.pack(inv_freq.data_ptr(), 2 * pairs, 1 if interleaved else 0, at, axes, stride_axis, stride_batch,
                      table_at), table


def _rope_apply(func, q, k, positions, inv_freq, pair_axis, interleaved, q_out, k_out, stream):
    if stream is not None:
        return _on_stream(_rope_apply, stream, q, func, q, k, positions, inv_freq, pair_axis, interleaved, q_out, k_out,
                          None)
    done = _fast().rope(func == "rope_bwd", q, k, positions, inv_freq, pair_axis, interleaved, q_out, k_out)
    if done is not None:
        if done.__class__ is int:
            _check(func, done)
        return done
    hq = _heads("q", q, None, 4)
    dev = q.device
    B, _, N, d = q.shape
    hk = None
    if k is not None:
        hk = _heads("k", k, dev, 4)
        if k.shape[0] != B or k.shape[2] != N or k.shape[3] != d:
            raise ValueError("k must be [B, Hk, N, d] matching q")
    rope, keep = _rope(inv_freq, positions, (B, N), pair_axis, interleaved, dev)
    outs, ho = [], []
    for name, x, out in (("q_out", q, q_out), ("k_out", k, k_out)):
        if x is None:
            if out is not None:
                raise ValueError("%s without its input" % name)
            outs.append(None)
            ho.append(None)
            continue
        if out is None:
            out = torch.empty(x.shape, dtype=torch.bfloat16, device=dev)
            H = x.shape[1]
            ho.append(_HEADS.pack(out.data_ptr(), H * N * d, d, N * d, H))
        else:
            ho.append(_heads(name, out, dev, 4))
            _need_shape(name, out, x.shape)
        outs.append(out)
    _call(func, dev, hq, hk, ho[0], ho[1], rope, B, N, d, _stream_handle(None, dev))
    del keep                                       # the library has read the axis table by now
    return tuple(outs)


def rope_fwd(q, k, positions, inv_freq, pair_axis=None, interleaved=False, q_out=None, k_out=None,
             stream=None):
    """Rotary positions on queries and keys.  q [B,Hq,N,d], k [B,Hk,N,d] (or
    None) bf16 with any strides but a contiguous last dimension, so a
    projection output [B,N,H*d] goes in as ``.view(B,N,H,d).transpose(1,2)``;
    inv_freq [rot/2] fp32; positions int32 [N] or [B,N], or, with ``pair_axis``
    (rot/2 axis numbers, e.g. 0 time, 1 height, 2 width), [axes,N] or
    [axes,B,N].

    Returns (q_out, k_out) bf16: new contiguous [B,H,N,d] tensors, as
    ``attn_fwd`` takes them, unless given (any strides; the inputs themselves
    for a rotation in place).
    """
    return _rope_apply("rope_fwd", q, k, positions, inv_freq, pair_axis, interleaved, q_out, k_out, stream)


def rope_bwd(dq_out, dk_out, positions, inv_freq, pair_axis=None, interleaved=False, dq=None, dk=None,
             stream=None):
    """Gradients of rope_fwd: from those of its outputs (dq_out [B,Hq,N,d],
    dk_out or None) to those of its inputs.  The other arguments are
    rope_fwd's.  Returns (dq, dk), new contiguous tensors unless given."""
    return _rope_apply("rope_bwd", dq_out, dk_out, positions, inv_freq, pair_axis, interleaved, dq, dk, stream)


def _token_map(block_table, seq_ids, positions, T, device):
    """Checks shared by the calls that address cached tokens one by one."""
    for name, t in (("block_table", block_table), ("seq_ids", seq_ids), ("positions", positions)):
        _need_cuda(name, t, torch.int32, device)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [num_seqs, max_blocks]")
    _need_shape("seq_ids", seq_ids, (T,))
    _need_shape("positions", positions, (T,))


def _append_args(q, k, v, block_table, seq_ids, positions, inv_freq, rope_positions, pair_axis, interleaved,
                 q_out):
    hk = _heads("k", k, None, 3)
    dev = k.device
    hv = _heads("v", v, dev, 3)
    if v.shape != k.shape:
        raise ValueError("k and v must have the same shape [T, Hkv, d]")
    T, _, d = k.shape
    _token_map(block_table, seq_ids, positions, T, dev)
    hq = ho = None
    if q is not None:
        hq = _heads("q", q, dev, 3)
        if q.shape[0] != T or q.shape[2] != d:
            raise ValueError("q must be [T, Hq, d] matching k")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
        ho = _heads("q_out", q_out, dev, 3)
        _need_shape("q_out", q_out, q.shape)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rope = (None, None)
    if inv_freq is not None:
        rope = _rope(inv_freq, rope_positions, (T,), pair_axis, interleaved, dev)
    elif rope_positions is not None or pair_axis is not None:
        raise ValueError("rope_positions and pair_axis need inv_freq")
    return dev, T, d, hq, hk, hv, ho, rope, q_out


def rope_append_paged(q, k, v, k_cache, v_cache, block_table, seq_ids, positions, inv_freq=None,
                      rope_positions=None, pair_axis=None, interleaved=False, q_out=None, stream=None):
    """A step's new tokens into the paged cache: queries rotated, keys rotated
    and stored, values stored, in one kernel.  q [T,Hq,d] (or None), k and v
    [T,Hkv,d] bf16, any strides but a contiguous last dimension; caches
    [num_blocks,Hkv,16,d] bf16 (updated in place); block_table
    [num_seqs,max_blocks], seq_ids [T] (negative: a padding row, nothing is
    done for it) and positions [T] int32: row t takes position positions[t] of
    sequence seq_ids[t].  inv_freq [rot/2] fp32 (None: no rotation);
    rope_positions [T], or with ``pair_axis`` [axes,T], where the rotation's
    positions are not the cache's.

    Returns q_out [T,Hq,d] (new unless given; its padding rows are left as
    they were), or None without q.
    """
    if stream is not None:
        return _on_stream(rope_append_paged, stream, k, q, k, v, k_cache, v_cache, block_table, seq_ids, positions, inv_freq,
                          rope_positions, pair_axis, interleaved, q_out)
    if v_cache is not None:                        # (None: a 4-bit cache)
        done = _fast().append(q, k, v, k_cache, v_cache, block_table, seq_ids, positions, 0, inv_freq, rope_positions,
                              pair_axis, interleaved, q_out)
        if done is not None:
            if done.__class__ is int:
                _check("rope_append_paged", done)
            return done[0]
    dev, T, d, hq, hk, hv, ho, rope, q_out = _append_args(
        q, k, v, block_table, seq_ids, positions, inv_freq, rope_positions, pair_axis, interleaved, q_out)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        _need_cuda(name, t, torch.bfloat16, dev)
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("caches must be [num_blocks,Hkv,block_size,d]")
    nb, Hkv, bs, dc = k_cache.shape
    if Hkv != k.shape[1] or dc != d:
        raise ValueError("caches must have k's heads and head dim")
    _call("rope_append_paged", dev, hq, hk, hv, ho, rope[0], _ptr(k_cache), _ptr(v_cache),
          _ptr(block_table), _ptr(seq_ids), _ptr(positions), T, block_table.shape[0], d, bs, block_table.shape[1], nb,
          _stream_handle(None, dev))
    return q_out


@functools.lru_cache(maxsize=None)
def kv4_record_bytes(d, group):
    """Bytes of one (block, KV head) record of a 4-bit cache."""
    n = int(load_library().kv4_record_bytes(int(d), int(group)))
    if n == 0:
        raise ValueError("a 4-bit cache has d 64 or 128 and groups of 32 or 64, got d %d, group %d" % (d, group))
    return n


def _need_kv4(kv_cache, d, group, device):
    """(num_blocks, Hkv) of a 4-bit cache."""
    _need_cuda("kv_cache", kv_cache, torch.uint8, device)
    shape = kv_cache.shape
    if len(shape) != 3 or shape[2] != kv4_record_bytes(d, group):
        raise ValueError("kv_cache must be [num_blocks, Hkv, %d] for d %d and group %d, got %s"
                         % (kv4_record_bytes(d, group), d, group, tuple(shape)))
    return shape[0], shape[1]


def rope_append_paged_kv4(q, k, v, kv_cache, block_table, seq_ids, positions, group, inv_freq=None,
                          rope_positions=None, pair_axis=None, interleaved=False, q_out=None, stream=None):
    """rope_append_paged into a 4-bit cache: kv_cache
    [num_blocks,Hkv,kv4_record_bytes(d, group)] uint8 (updated in place), 4-bit
    codes with a bf16 (min, scale) per ``group`` (32 or 64) consecutive
    elements of a key or value.  Returns q_out (or None without q)."""
    if stream is not None:
        return _on_stream(rope_append_paged_kv4, stream, k, q, k, v, kv_cache, block_table, seq_ids, positions, group,
                          inv_freq, rope_positions, pair_axis, interleaved, q_out)
    done = _fast().append(q, k, v, kv_cache, None, block_table, seq_ids, positions, group, inv_freq, rope_positions,
                          pair_axis, interleaved, q_out)
    if done is not None:
        if done.__class__ is int:
            _check("rope_append_paged_kv4", done)
        return done[0]
    dev, T, d, hq, hk, hv, ho, rope, q_out = _append_args(
        q, k, v, block_table, seq_ids, positions, inv_freq, rope_positions, pair_axis, interleaved, q_out)
    nb, Hkv = _need_kv4(kv_cache, d, group, dev)
    if Hkv != k.shape[1]:
        raise ValueError("kv_cache must have k's heads")
    _call("rope_append_paged_kv4", dev, hq, hk, hv, ho, rope[0], _ptr(kv_cache), group,
          _ptr(block_table), _ptr(seq_ids), _ptr(positions), T, block_table.shape[0], d, BLOCK_SIZE,
          block_table.shape[1], nb, _stream_handle(None, dev))
    return q_out


def kv4_read_paged(kv_cache, block_table, seq_ids, positions, d, group, k=None, v=None, stream=None):
    """The values that cached tokens of a 4-bit cache stand for: row t is
    position positions[t] of sequence seq_ids[t] ([T] int32; negative
    sequences: rows left as they were).  Returns (k, v) [T,Hkv,d] bf16, which
    rope_append_paged puts into a bf16 cache (for attn_prefill_paged, say)."""
    if stream is not None:
        return _on_stream(kv4_read_paged, stream, kv_cache, kv_cache, block_table, seq_ids, positions, d, group, k, v)
    done = _fast().read(kv_cache, block_table, seq_ids, positions, d, group, k, v)
    if done is not None:
        if done.__class__ is int:
            _check("kv4_read_paged", done)
        return done
    if not isinstance(seq_ids, torch.Tensor) or seq_ids.dim() != 1:
        raise ValueError("seq_ids must be a [T] tensor")
    nb, Hkv = _need_kv4(kv_cache, d, group, None)
    dev, T = kv_cache.device, seq_ids.shape[0]
    _token_map(block_table, seq_ids, positions, T, dev)
    k = _output("k", k, (T, Hkv, d), torch.bfloat16, dev)
    v = _output("v", v, (T, Hkv, d), torch.bfloat16, dev)
    _call("kv4_read_paged", dev, _ptr(kv_cache), group, _ptr(block_table), _ptr(seq_ids), _ptr(positions), _ptr(k),
          _ptr(v), T, block_table.shape[0], Hkv, d, BLOCK_SIZE, block_table.shape[1], nb, _stream_handle(None, dev))
    return k, v


@functools.lru_cache(maxsize=None)
def kv8_record_bytes(d):
    """Bytes of one (block, KV head) record of an 8-bit cache."""
    n = int(load_library().kv8_record_bytes(int(d)))
    if n == 0:
        raise ValueError("an 8-bit cache has d 64 or 128, got d %d" % d)
    return n


def _need_kv8(kv_cache, d, device):
    """(num_blocks, Hkv) of an 8-bit cache."""
    _need_cuda("kv_cache", kv_cache, torch.uint8, device)
    shape = kv_cache.shape
    if len(shape) != 3 or shape[2] != kv8_record_bytes(d):
        raise ValueError("kv_cache must be [num_blocks, Hkv, %d] for d %d, got %s"
                         % (kv8_record_bytes(d), d, tuple(shape)))
    return shape[0], shape[1]


def kv8_append_paged(q, k, v, kv_cache, block_table, seq_ids, positions, inv_freq=None, rope_positions=None,
                     pair_axis=None, interleaved=False, q_out=None, stream=None):
    """rope_append_paged into an 8-bit cache: kv_cache
    [num_blocks,Hkv,kv8_record_bytes(d)] uint8 (updated in place), e4m3 codes
    with a scale (a power of two) per block of 16 tokens and head for the keys
    and one for the values.  Rows that fall into one block stand together, in
    ascending order of their positions (some may be left out); a row for a
    block's first slot begins it anew.
    Returns q_out (or None without q)."""
    if stream is not None:
        return _on_stream(kv8_append_paged, stream, k, q, k, v, kv_cache, block_table, seq_ids, positions,
                          inv_freq, rope_positions, pair_axis, interleaved, q_out)
    done = _fast().append8(q, k, v, kv_cache, None, block_table, seq_ids, positions, 0, inv_freq, rope_positions,
                           pair_axis, interleaved, q_out)
    if done is not None:
        if done.__class__ is int:
            _check("kv8_append_paged", done)
        return done[0]
    dev, T, d, hq, hk, hv, ho, rope, q_out = _append_args(
        q, k, v, block_table, seq_ids, positions, inv_freq, rope_positions, pair_axis, interleaved, q_out)
    nb, Hkv = _need_kv8(kv_cache, d, dev)
    if Hkv != k.shape[1]:
        raise ValueError("kv_cache must have k's heads")
    _call("kv8_append_paged", dev, hq, hk, hv, ho, rope[0], _ptr(kv_cache), _ptr(block_table), _ptr(seq_ids),
          _ptr(positions), T, block_table.shape[0], d, BLOCK_SIZE, block_table.shape[1], nb,
          _stream_handle(None, dev))
    return q_out


def kv8_read_paged(kv_cache, block_table, seq_ids, positions, d, k=None, v=None, stream=None):
    """The values that cached tokens of an 8-bit cache stand for: row t is
    position positions[t] of sequence seq_ids[t] ([T] int32; negative
    sequences: rows left as they were).  Returns (k, v) [T,Hkv,d] bf16."""
    if stream is not None:
        return _on_stream(kv8_read_paged, stream, kv_cache, kv_cache, block_table, seq_ids, positions, d, k, v)
    done = _fast().read8(kv_cache, block_table, seq_ids, positions, d, 0, k, v)
    if done is not None:
        if done.__class__ is int:
            _check("kv8_read_paged", done)
        return done
    if not isinstance(seq_ids, torch.Tensor) or seq_ids.dim() != 1:
        raise ValueError("seq_ids must be a [T] tensor")
    nb, Hkv = _need_kv8(kv_cache, d, None)
    dev, T = kv_cache.device, seq_ids.shape[0]
    _token_map(block_table, seq_ids, positions, T, dev)
    k = _output("k", k, (T, Hkv, d), torch.bfloat16, dev)
    v = _output("v", v, (T, Hkv, d), torch.bfloat16, dev)
    _call("kv8_read_paged", dev, _ptr(kv_cache), _ptr(block_table), _ptr(seq_ids), _ptr(positions), _ptr(k), _ptr(v),
          T, block_table.shape[0], Hkv, d, BLOCK_SIZE, block_table.shape[1], nb, _stream_handle(None, dev))
    return k, v


@functools.lru_cache(maxsize=1024)
def attn_decode_paged_kv4_workspace_size(num_seqs, Hq, Hkv, d):
    return int(load_library().attn_decode_paged_kv4_workspace_size(num_seqs, Hq, Hkv, d))


def attn_decode_paged_kv4(q, kv_cache, block_table, seq_lens, group, scale=None, o=None, lse=None,
                          workspace=None, return_lse=True, stream=None):
    """attn_decode_paged over a 4-bit cache.  q [S,Hq,d] bf16; kv_cache
    [num_blocks,Hkv,kv4_record_bytes(d, group)] uint8; block_table
    [S,max_blocks] int32; seq_lens [S] int32 (all on the GPU).

    Returns (o [S,Hq,d] bf16, lse [S,Hq] fp32 or None).
    """
    if stream is not None:
        return _on_stream(attn_decode_paged_kv4, stream, q, q, kv_cache, block_table, seq_lens, group, scale, o, lse,
                          workspace, return_lse)
    done = _fast().decode(q, kv_cache, block_table, seq_lens, group, scale, o, lse, workspace, return_lse)
    if done is not None:
        if done.__class__ is int:
            _check("attn_decode_paged_kv4", done)
        return done
    _need_cuda("q", q, torch.bfloat16)
    dev = q.device
    if q.dim() != 3:
        raise ValueError("q must be [S,Hq,d]")
    S, Hq, d = q.shape
    nb, Hkv = _need_kv4(kv_cache, d, group, dev)
    _need_cuda("block_table", block_table, torch.int32, dev)
    _need_cuda("seq_lens", seq_lens, torch.int32, dev)
    table_shape = block_table.shape
    if len(table_shape) != 2 or table_shape[0] != S:
        raise ValueError("block_table must be [S, max_blocks]")
    _need_shape("seq_lens", seq_lens, (S,))
    o = _output("o", o, (S, Hq, d), torch.bfloat16, dev)
    if lse is not None or return_lse:
        lse = _output("lse", lse, (S, Hq), torch.float32, dev)
    if scale is None:
        scale = d ** -0.5
    workspace = _workspace("workspace", workspace, attn_decode_paged_kv4_workspace_size(S, Hq, Hkv, d), dev)
    _call("attn_decode_paged_kv4", dev, _ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens), S, Hq, Hkv, d,
          group, BLOCK_SIZE, table_shape[1], nb, float(scale), _ptr(o), _ptr(lse), _ptr(workspace),
          workspace.numel() * workspace.element_size(), _stream_handle(None, dev))
    return o, lse


@functools.lru_cache(maxsize=1024)
def attn_decode_paged_kv8_workspace_size(num_seqs, Hq, Hkv, d):
    return int(load_library().attn_decode_paged_kv8_workspace_size(num_seqs, Hq, Hkv, d))


@functools.lru_cache(maxsize=1024)
def attn_prefill_paged_kv8_workspace_size(num_seqs, Hq, Hkv, N, d):
    return int(load_library().attn_prefill_paged_kv8_workspace_size(num_seqs, Hq, Hkv, N, d))


def _attend_kv8(func, q, kv_cache, block_table, seq_lens, scale, o, lse, workspace, return_lse):
    """Both attentions over an 8-bit cache, the longer way: q [S,Hq,d] or
    [S,Hq,N,d]."""
    _need_cuda("q", q, torch.bfloat16)
    dev = q.device
    if func == "attn_decode_paged_kv8":
        if q.dim() != 3:
            raise ValueError("q must be [S,Hq,d]")
        S, Hq, d = q.shape
        rows, size = (), attn_decode_paged_kv8_workspace_size
    else:
        if q.dim() != 4:
            raise ValueError("q must be [S,Hq,N,d]")
        S, Hq, N, d = q.shape
        rows, size = (N,), attn_prefill_paged_kv8_workspace_size
    nb, Hkv = _need_kv8(kv_cache, d, dev)
    _need_cuda("block_table", block_table, torch.int32, dev)
    _need_cuda("seq_lens", seq_lens, torch.int32, dev)
    table_shape = block_table.shape
    if len(table_shape) != 2 or table_shape[0] != S:
        raise ValueError("block_table must be [S, max_blocks]")
    _need_shape("seq_lens", seq_lens, (S,))
    o = _output("o", o, q.shape, torch.bfloat16, dev)
    if lse is not None or return_lse:
        lse = _output("lse", lse, q.shape[:-1], torch.float32, dev)
    if scale is None:
        scale = d ** -0.5
    workspace = _workspace("workspace", workspace, size(S, Hq, Hkv, *rows, d), dev)
    _call(func, dev, _ptr(q), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens), S, Hq, Hkv, *rows, d, BLOCK_SIZE,
          table_shape[1], nb, float(scale), _ptr(o), _ptr(lse), _ptr(workspace),
          workspace.numel() * workspace.element_size(), _stream_handle(None, dev))
    return o, lse


def attn_decode_paged_kv8(q, kv_cache, block_table, seq_lens, scale=None, o=None, lse=None, workspace=None,
                          return_lse=True, stream=None):
    """attn_decode_paged over an 8-bit cache.  q [S,Hq,d] bf16; kv_cache
    [num_blocks,Hkv,kv8_record_bytes(d)] uint8; block_table [S,max_blocks]
    int32; seq_lens [S] int32 (all on the GPU).

    Returns (o [S,Hq,d] bf16, lse [S,Hq] fp32 or None).
    """
    if stream is not None:
        return _on_stream(attn_decode_paged_kv8, stream, q, q, kv_cache, block_table, seq_lens, scale, o, lse,
                          workspace, return_lse)
    done = _fast().decode8(q, kv_cache, block_table, seq_lens, 0, scale, o, lse, workspace, return_lse)
    if done is not None:
        if done.__class__ is int:
            _check("attn_decode_paged_kv8", done)
        return done
    return _attend_kv8("attn_decode_paged_kv8", q, kv_cache, block_table, seq_lens, scale, o, lse, workspace, return_lse)


def attn_prefill_paged_kv8(q, kv_cache, block_table, seq_lens, scale=None, o=None, lse=None, workspace=None,
                           return_lse=True, stream=None):
    """The last N tokens of each sequence attend to an 8-bit cache that holds
    them already (see kv8_append_paged): a prompt's chunk, or draft tokens.
    q [S,Hq,N,d] bf16: query i is the token at position seq_lens[b] - N + i and
    sees the keys up to itself (before position 0: none, o = 0 and lse = -inf);
    the other arguments are attn_decode_paged_kv8's.

    Returns (o [S,Hq,N,d] bf16, lse [S,Hq,N] fp32 or None).
    """
    if stream is not None:
        return _on_stream(attn_prefill_paged_kv8, stream, q, q, kv_cache, block_table, seq_lens, scale, o, lse,
                          workspace, return_lse)
    done = _fast().prefill8(q, kv_cache, block_table, seq_lens, 0, scale, o, lse, workspace, return_lse)
    if done is not None:
        if done.__class__ is int:
            _check("attn_prefill_paged_kv8", done)
        return done
    return _attend_kv8("attn_prefill_paged_kv8", q, kv_cache, block_table, seq_lens, scale, o, lse, workspace,
                       return_lse)


def device_status(stream=None):
    """Read and clear the device status word (ATTN_DEV_* bits)."""
    flags = ctypes.c_uint(0)
    _check("attn_get_device_status",
           load_library().attn_get_device_status(_stream_handle(stream), ctypes.byref(flags)))
    return int(flags.value)


def set_wait_timeout_ns(ns):
    load_library().attn_set_wait_timeout_ns(int(ns))


def set_decode_max_ctas(ctas):
    """Cap the CTAs of a decode launch (0: one full wave)."""
    load_library().attn_set_decode_max_ctas(int(ctas))


def set_decode_early_plan(on):
    """Let later decode calls read seq_lens and block_table (``on`` = 1 or
    True), and also the first cache blocks of each CTA's share except a
    sequence's last block (``on`` = 2), before the preceding kernel in the
    stream has finished; the caller guarantees that kernel writes none of
    them.  0 or False: read nothing before it has finished."""
    level = int(on)
    load_library().attn_set_decode_early_plan(0 if level <= 0 else 2 if level >= 2 else 1)


def selftest_exp2_poly(x, y=None, stream=None):
    """y = 2^x (fp32 CUDA tensors) by the forward softmax's FMA-pipe exp2."""
    _need_cuda("x", x, torch.float32)
    dev = x.device
    y = _output("y", y, x.shape, torch.float32, dev)
    _call("attn_selftest_exp2_poly", dev, _ptr(x), _ptr(y), x.numel(), _stream_handle(stream, dev))
    return y


def selftest_wait_timeout(timeout_ns, stream=None):
    flags = ctypes.c_uint(0)
    _check("attn_selftest_wait_timeout",
           load_library().attn_selftest_wait_timeout(int(timeout_ns), _stream_handle(stream),
                                                     ctypes.byref(flags)))
    return int(flags.value)


def abi_version():
    return int(load_library().attn_abi_version())
