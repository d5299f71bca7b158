"""Python binding of the paged-KV calls of libspecverify.so (``include/spec_kv.h``):
``kv_blocktable_extend``, ``kv_cache_append`` and ``kv_paged_attention``.

As in the package's other calls, tensors are checked for device, dtype, shape
and layout, and their pointers go to the C ABI on torch's current stream of
their device; every call is asynchronous.  Inference only: no call records a
gradient.
"""

import ctypes
import sys

import torch

_pkg = sys.modules[__package__]      # the package, whose library() is the loaded build

SV_DTYPE_F16 = 2
MAX_HEAD_DIM = 256

# Every symbol include/spec_kv.h declares.
KV_EXPORTED = ("spec_kv_abi_version", "kv_blocktable_extend", "kv_cache_append",
               "kv_paged_attention_workspace_bytes", "kv_paged_attention")

_I32_MAX = 0x7fffffff
_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: SV_DTYPE_F16}


class AppendDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("block_stride", ctypes.c_int64)]


class AttentionDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("sliding_window", ctypes.c_int32),
                ("max_new", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("q_stride", ctypes.c_int64), ("block_stride", ctypes.c_int64),
                ("scale", ctypes.c_float), ("reserved_f", ctypes.c_float)]


def set_signatures(lib):
    """Entry-point signatures of include/spec_kv.h on a loaded library."""
    P, i32 = ctypes.c_void_p, ctypes.c_int32
    lib.spec_kv_abi_version.restype = i32
    lib.kv_blocktable_extend.restype = i32
    lib.kv_blocktable_extend.argtypes = [i32, i32, i32, P, P, P, P, i32, P, P, i32, P, i32, P, P,
                                         P, P, P, P, P]
    lib.kv_cache_append.restype = i32
    lib.kv_cache_append.argtypes = [ctypes.POINTER(AppendDesc), P, P, P, P, P, P]
    lib.kv_paged_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.kv_paged_attention_workspace_bytes.argtypes = [ctypes.POINTER(AttentionDesc)]
    lib.kv_paged_attention.restype = i32
    lib.kv_paged_attention.argtypes = [ctypes.POINTER(AttentionDesc), P, P, P, P, P, P, P, P, P,
                                       ctypes.c_size_t, P]


def _call(fn, index, *args):
    """Calls an entry point on torch's current stream of GPU ``index``, with that
    device current (the null stream belongs to the current device)."""
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        _pkg._check(status)


def _gpu(t):
    """The device index of a GPU tensor."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a GPU")
    return t.get_device()


def _tensor(t, name, dtype, shape, index):
    """The pointer of a contiguous tensor of this dtype and shape on GPU ``index``."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or \
            t.get_device() != index:
        raise ValueError(f"{name} must be a contiguous {str(dtype)[6:]} tensor of shape "
                         f"{list(shape)} on cuda:{index}, got {str(t.dtype)[6:]} "
                         f"{list(t.shape)} on {t.device}")
    return t.data_ptr()


def _i32(value, name):
    """An argument of the C ABI's 32-bit type (ctypes would cut it to size)."""
    value = int(value)
    if not -_I32_MAX - 1 <= value <= _I32_MAX:
        raise ValueError(f"{name} must be a 32-bit integer, got {value}")
    return value


def _caches(k_cache, v_cache, dtype, index):
    """(blocks, kv_heads, block_size, head_dim, block stride) of a cache pair on
    device ``index`` (-1: the host)."""
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must both be [num_blocks, kv_heads, block_size, "
                         "head_dim]")
    nb, kv, bs, dim = shape
    if k_cache.dtype is not dtype or v_cache.dtype is not dtype or \
            k_cache.get_device() != index or v_cache.get_device() != index:
        raise ValueError(f"k_cache and v_cache must have the rows' dtype ({str(dtype)[6:]}) and "
                         "device")
    sk, sv = k_cache.stride(), v_cache.stride()
    for name, s in (("k_cache", sk), ("v_cache", sv)) if sk != sv else (("k_cache", sk),):
        # strides of dimensions of size 1 say nothing
        if (dim > 1 and s[3] != 1) or (bs > 1 and s[2] != dim) or (kv > 1 and s[1] != bs * dim):
            raise ValueError(f"{name}: each block must be contiguous")
    if nb <= 1:
        return nb, kv, bs, dim, 0
    if sk[0] != sv[0]:
        raise ValueError("k_cache and v_cache must have one block stride")
    if sk[0] < kv * bs * dim:                   # (an expanded cache has 0)
        raise ValueError("the blocks of a cache must not overlap")
    return nb, kv, bs, dim, sk[0]


def _row_stride(t, name):
    """Elements between the token rows of [T, heads, dim] with contiguous heads
    (0: a single row leaves it open)."""
    s = t.stride()
    if len(s) != 3:
        raise ValueError(f"{name} must be [T, heads, head_dim]")
    T, heads, dim = t.shape
    if (dim > 1 and s[2] != 1) or (heads > 1 and s[1] != dim):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    if T <= 1:
        return 0
    if s[0] < heads * dim:                      # (an expanded row has 0)
        raise ValueError(f"{name}: the token rows must not overlap")
    return s[0]


def kv_blocktable_extend(block_table, seq_lens, num_new, free_blocks, free_count, block_size,
                         max_tokens, *, freed_blocks=None, num_freed=None, out=None):
    """Blocks and slots for ``num_new`` [B] more tokens per sequence.

    Takes ids from the end of the stack ``free_blocks[:free_count]`` (after
    pushing ``freed_blocks`` [B, max_freed] / ``num_freed`` [B] as
    ``kv_blocktable_truncate`` returns them; ids that ``free_blocks`` has no room
    for are dropped, so give it room for every block of the cache), writes them to ``block_table``
    [B, max_blocks] in place, and returns a dict of device tensors: new_lens
    [B], num_taken [B] (-1: bad request, -2: pool short; such sequences stay
    as they were), free_left [1], cu_tokens [B+1], slot_map [max_tokens] int64
    and positions [max_tokens] (-1 where there is no token).  ``max_tokens``:
    rows of the packed token arrays, at least the sum of num_new.  ``out``: a
    dict of an earlier call of the same shape, whose tensors are reused; its
    new_lens may be ``seq_lens`` and its free_left ``free_count``."""
    lib = _pkg.library()
    dev, i32 = _gpu(block_table), torch.int32      # dev: its index
    B, width = block_table.shape
    T = _i32(max_tokens, "max_tokens")
    if T < 0:
        raise ValueError("max_tokens must not be negative")
    p = (_tensor(block_table, "block_table", i32, (B, width), dev),
         _tensor(seq_lens, "seq_lens", i32, (B,), dev),
         _tensor(num_new, "num_new", i32, (B,), dev),
         _tensor(free_blocks, "free_blocks", i32, (free_blocks.numel(),), dev))
    pc = _tensor(free_count, "free_count", i32, (1,), dev)
    pf = pn = None
    max_freed = 0
    if freed_blocks is not None:
        if num_freed is None:
            raise ValueError("freed_blocks needs num_freed")
        if freed_blocks.dim() != 2:
            raise ValueError("freed_blocks must be [B, max_freed]")
        max_freed = freed_blocks.shape[1]
        pf = _tensor(freed_blocks, "freed_blocks", i32, (B, max_freed), dev) if max_freed else None
        pn = _tensor(num_freed, "num_freed", i32, (B,), dev)
    if out is None:
        on = dict(dtype=i32, device=block_table.device)
        out = dict(new_lens=torch.empty(B, **on), num_taken=torch.empty(B, **on),
                   free_left=torch.empty(1, **on), cu_tokens=torch.empty(B + 1, **on),
                   slot_map=torch.empty(T, dtype=torch.int64, device=block_table.device),
                   positions=torch.empty(T, **on))
    _call(lib.kv_blocktable_extend, dev, B, width, _i32(block_size, "block_size"), p[0], p[1], p[2], p[3],
          free_blocks.numel(), pc, pf, max_freed, pn, T,
          _tensor(out["new_lens"], "out new_lens", i32, (B,), dev),
          _tensor(out["num_taken"], "out num_taken", i32, (B,), dev),
          _tensor(out["free_left"], "out free_left", i32, (1,), dev),
          _tensor(out["cu_tokens"], "out cu_tokens", i32, (B + 1,), dev),
          _tensor(out["slot_map"], "out slot_map", torch.int64, (T,), dev),
          _tensor(out["positions"], "out positions", i32, (T,), dev))
    return out


def kv_cache_append(k, v, slot_map, k_cache, v_cache):
    """Writes the rows of ``k`` and ``v`` [T, kv_heads, head_dim] (parts of wider
    rows allowed) to their slots of the caches [num_blocks, kv_heads, block_size,
    head_dim] in place.  ``slot_map`` [T] int64: negative or out-of-cache slots
    skip their row; the others must differ.  Float32, bfloat16 or float16."""
    lib = _pkg.library()
    code = _CODES.get(k.dtype)
    if code is None:
        raise TypeError(f"k must be float32, bfloat16 or float16, got {k.dtype}")
    dev = _gpu(k)
    nb, kv, bs, dim, block_stride = _caches(k_cache, v_cache, k.dtype, dev)
    shape = k.shape
    if shape[1:] != (kv, dim) or v.shape != shape or v.dtype is not k.dtype or \
            v.get_device() != dev:
        raise ValueError(f"k and v must be [T, {kv}, {dim}] of one dtype on one device")
    T = shape[0]
    if max(T, nb) > _I32_MAX:
        raise ValueError(f"T and num_blocks must be 32-bit integers, got {T} and {nb}")
    desc = AppendDesc(T, kv, dim, bs, nb, code, _row_stride(k, "k"), _row_stride(v, "v"),
                      block_stride)
    _call(lib.kv_cache_append, dev, ctypes.byref(desc), k.data_ptr(), v.data_ptr(),
          _tensor(slot_map, "slot_map", torch.int64, (T,), dev), k_cache.data_ptr(),
          v_cache.data_ptr())


def _attention_desc(q, k_cache, v_cache, block_table, scale, sliding_window, max_new):
    code = _CODES.get(q.dtype)
    if code is None:
        raise TypeError(f"q must be float32, bfloat16 or float16, got {q.dtype}")
    nb, kv, bs, dim, block_stride = _caches(k_cache, v_cache, q.dtype, q.get_device())
    stride = _row_stride(q, "q")
    T, heads, q_dim = q.shape
    if q_dim != dim:
        raise ValueError(f"q must be [T, heads, {dim}]")
    B, width = block_table.shape
    if max(T, nb, sliding_window, max_new) > _I32_MAX or min(sliding_window, max_new) < 0:
        for name, value in (("T", T), ("num_blocks", nb), ("sliding_window", sliding_window),
                            ("max_new", max_new)):
            _i32(value, name)
    return AttentionDesc(B, T, heads, kv, dim, bs, nb, width, code, int(sliding_window),
                         int(max_new), 0, stride, block_stride,
                         dim ** -0.5 if scale is None else float(scale), 0.0)


def kv_paged_attention_workspace_bytes(q, k_cache, v_cache, block_table, *, sliding_window=0,
                                       max_new=0):
    """Workspace bytes of ``kv_paged_attention`` on tensors of these shapes."""
    desc = _attention_desc(q, k_cache, v_cache, block_table, None, sliding_window, max_new)
    return int(_pkg.library().kv_paged_attention_workspace_bytes(ctypes.byref(desc)))


def kv_paged_attention(q, k_cache, v_cache, block_table, seq_lens, cu_tokens, *, scale=None,
                       sliding_window=0, max_new=0, lse=False, out=None, workspace=None):
    """Causal attention of each sequence's last tokens over its pages.

    ``q`` [T, heads, head_dim] (rows of a wider projection allowed) holds the
    queries of sequence b in rows cu_tokens[b] .. cu_tokens[b+1]-1, its last
    tokens of ``seq_lens`` [B]; their keys and values are in the caches
    [num_blocks, kv_heads, block_size, head_dim] already, found through
    ``block_table`` [B, max_blocks].  ``scale`` defaults to head_dim^-0.5;
    ``sliding_window`` W > 0 lets a token see itself and the W - 1 before it;
    ``max_new``, the most new tokens of a sequence (0: the batch's mean is taken),
    picks the tile shape only.  Returns dict(out [T, heads, head_dim], lse
    [T, heads] float32 or None, workspace).  ``out``: a dict of an earlier call of
    the same shape, whose tensors are reused; a call with another ``max_new`` or
    ``sliding_window`` that needs a larger workspace puts one there.  An explicit
    ``workspace`` has to be large enough.  Rows of no sequence are left as they
    were."""
    lib = _pkg.library()
    desc = _attention_desc(q, k_cache, v_cache, block_table, scale, sliding_window, max_new)
    dev = _gpu(q)
    B, T, heads, dim = desc.batch, desc.tokens, desc.heads, desc.head_dim
    pt = _tensor(block_table, "block_table", torch.int32, (B, desc.max_blocks), dev)
    pl = _tensor(seq_lens, "seq_lens", torch.int32, (B,), dev)
    pc = _tensor(cu_tokens, "cu_tokens", torch.int32, (B + 1,), dev)
    if out is None:
        out = dict(out=torch.empty((T, heads, dim), dtype=q.dtype, device=q.device),
                   lse=torch.empty((T, heads), dtype=torch.float32, device=q.device)
                   if lse else None, workspace=None)
    elif lse and out["lse"] is None:
        raise ValueError("out holds no lse tensor")
    kept = workspace is None      # out's own, which another hint or window may have sized
    if kept:
        workspace = out["workspace"]
    if workspace is None:
        need = lib.kv_paged_attention_workspace_bytes(ctypes.byref(desc))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on q's device")
    out["workspace"] = workspace
    tensors = (ctypes.byref(desc), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), pt, pl, pc,
               _tensor(out["out"], "out", q.dtype, (T, heads, dim), dev),
               _tensor(out["lse"], "out lse", torch.float32, (T, heads), dev)
               if out["lse"] is not None else None)
    try:
        _call(lib.kv_paged_attention, dev, *tensors,
              workspace.data_ptr() if workspace is not None else None,
              workspace.numel() * workspace.element_size() if workspace is not None else 0)
    except _pkg.SpecVerifyError as e:
        if not kept or e.status != _pkg.SV_ERR_WORKSPACE:
            raise
        # a larger one takes its place and keeps it: a captured call may still use it
        need = lib.kv_paged_attention_workspace_bytes(ctypes.byref(desc))
        larger = torch.empty(need, dtype=torch.uint8, device=q.device)
        larger.replaces = workspace
        out["workspace"] = larger
        _call(lib.kv_paged_attention, dev, *tensors, larger.data_ptr(), need)
    return out
