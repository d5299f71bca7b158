"""Python binding of the paged-KV calls of libspecverify.so (``include/spec_kv.h``):
``kv_blocktable_extend``, ``kv_cache_append``, ``kv_cache_append_rotary`` and
``kv_paged_attention``, and the cache held in 4 bits: ``make_kv_cache_q4``,
``kv_cache_append_q4``, ``kv_cache_read_q4`` and ``kv_paged_attention_q4``.

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
               "kv_paged_attention_workspace_bytes", "kv_paged_attention",
               "kv_cache_append_rotary", "kv_cache_append_q4", "kv_cache_read_q4",
               "kv_paged_attention_q4_workspace_bytes", "kv_paged_attention_q4")

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


class RotaryDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("table_rows", ctypes.c_int32),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64),
                ("block_stride", ctypes.c_int64)]


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
    lib.kv_cache_append_rotary.restype = i32
    lib.kv_cache_append_rotary.argtypes = [ctypes.POINTER(RotaryDesc)] + [P] * 10
    lib.kv_cache_append_q4.restype = i32
    lib.kv_cache_append_q4.argtypes = [ctypes.POINTER(RotaryDesc)] + [P] * 12
    lib.kv_cache_read_q4.restype = i32
    lib.kv_cache_read_q4.argtypes = [i32] * 6 + [P] * 8
    lib.kv_paged_attention_q4_workspace_bytes.restype = ctypes.c_size_t
    lib.kv_paged_attention_q4_workspace_bytes.argtypes = [ctypes.POINTER(AttentionDesc)]
    lib.kv_paged_attention_q4.restype = i32
    lib.kv_paged_attention_q4.argtypes = [ctypes.POINTER(AttentionDesc)] + [P] * 11 + \
        [ctypes.c_size_t, P]


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
    return _attend(lib.kv_paged_attention, lib.kv_paged_attention_workspace_bytes, desc, q,
                   (k_cache.data_ptr(), v_cache.data_ptr()), block_table, seq_lens, cu_tokens, lse,
                   out, workspace)


def _attend(call, workspace_bytes, desc, q, caches, block_table, seq_lens, cu_tokens, lse, out,
            workspace):
    """An attention call on caches of either kind (``caches``: their pointers)."""
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
        need = workspace_bytes(ctypes.byref(desc))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on q's device")
    out["workspace"] = workspace
    tensors = (ctypes.byref(desc), q.data_ptr(), *caches, pt, pl, pc,
               _tensor(out["out"], "out", q.dtype, (T, heads, dim), dev),
               _tensor(out["lse"], "out lse", torch.float32, (T, heads), dev)
               if out["lse"] is not None else None)
    try:
        _call(call, dev, *tensors,
              workspace.data_ptr() if workspace is not None else None,
              workspace.numel() * workspace.element_size() if workspace is not None else 0)
    except _pkg.SpecVerifyError as e:
        if not kept or e.status != _pkg.SV_ERR_WORKSPACE:
            raise
        # a larger one takes its place and keeps it: a captured call may still use it
        need = workspace_bytes(ctypes.byref(desc))
        larger = torch.empty(need, dtype=torch.uint8, device=q.device)
        larger.replaces = workspace
        out["workspace"] = larger
        _call(call, dev, *tensors, larger.data_ptr(), need)
    return out


def _rotation(desc, q, positions, cos_sin, interleaved, out, dev):
    """Fills in the rotation's part of a RotaryDesc; the pointers of q, positions,
    cos_sin and q_out, and the tensor of the last."""
    T = desc.tokens
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [positions, rotary_dim]")
    rows, rot = cos_sin.shape
    desc.rotary_dim, desc.table_rows = rot, _i32(rows, "the rows of cos_sin")
    desc.interleaved = 1 if interleaved else 0
    pc = _tensor(cos_sin, "cos_sin", torch.float32, (rows, rot), dev)
    pp = _tensor(positions, "positions", torch.int32, (T,), dev)
    if q is None:
        if out is not None:
            raise ValueError("out needs q")
        return None, pp, pc, None, None
    desc.q_stride = _row_stride(q, "q")
    if q.shape[0] != T or q.shape[2] != desc.head_dim or _CODES.get(q.dtype) != desc.dtype or \
            q.get_device() != dev:
        raise ValueError(f"q must be [{T}, heads, {desc.head_dim}] of the rows' dtype and device")
    desc.heads = q.shape[1]
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif out.shape != q.shape or out.dtype is not q.dtype or out.get_device() != dev:
        raise ValueError("out must have q's shape, dtype and device")
    desc.q_out_stride = _row_stride(out, "out")
    return q.data_ptr(), pp, pc, out.data_ptr(), out


def _row_desc(k, v, kv, bs, nb, dim, dev):
    """A RotaryDesc of key and value rows [T, kv, dim], without a rotation."""
    code = _CODES.get(k.dtype)
    if code is None:
        raise TypeError(f"k must be float32, bfloat16 or float16, got {k.dtype}")
    shape = k.shape
    if shape[1:] != (kv, dim) or v.shape != shape or v.dtype is not k.dtype or \
            v.get_device() != dev or k.get_device() != dev:
        raise ValueError(f"k and v must be [T, {kv}, {dim}] of one dtype on one device")
    T = shape[0]
    if max(T, nb) > _I32_MAX:
        raise ValueError(f"T and num_blocks must be 32-bit integers, got {T} and {nb}")
    return RotaryDesc(T, 0, kv, dim, bs, nb, code, 0, 0, 0, 0, _row_stride(k, "k"),
                      _row_stride(v, "v"), 0, 0)


def kv_cache_append_rotary(q, k, v, positions, cos_sin, slot_map, k_cache, v_cache, *,
                           interleaved=False, out=None):
    """``kv_cache_append`` with the position rotation on the way: the queries ``q``
    [T, heads, head_dim] (or None) and keys of each token are turned by the angles of its
    position, the keys and values written to their slots in place.

    ``positions`` [T] int32 (``kv_blocktable_extend``'s) picks a row of ``cos_sin``
    [positions, rotary_dim] float32: the cosines of its angles, then their sines.
    Channel i turns with i + rotary_dim / 2, or, ``interleaved``, 2i with 2i + 1;
    channels behind rotary_dim stay as they are.  Returns the turned queries: ``out``
    (which may be ``q`` itself, and overlaps it in no other way), or a new tensor.  Rows
    whose position is not in the table are skipped (their queries left as they were in
    ``out``), rows without a slot turn their query alone."""
    lib = _pkg.library()
    dev = _gpu(k)
    nb, kv, bs, dim, block_stride = _caches(k_cache, v_cache, k.dtype, dev)
    desc = _row_desc(k, v, kv, bs, nb, dim, dev)
    desc.block_stride = block_stride
    pq, pp, pc, po, out = _rotation(desc, q, positions, cos_sin, interleaved, out, dev)
    _call(lib.kv_cache_append_rotary, dev, ctypes.byref(desc), pq, k.data_ptr(), v.data_ptr(), pp, pc,
          _tensor(slot_map, "slot_map", torch.int64, (desc.tokens,), dev), po, k_cache.data_ptr(),
          v_cache.data_ptr())
    return out


def make_kv_cache_q4(num_blocks, kv_heads, block_size, head_dim, device="cuda"):
    """An empty paged cache held in 4 bits (head_dim a multiple of 32 up to 256):
    dict(k_codes, v_codes [num_blocks, kv_heads, block_size, head_dim / 2] uint8,
    k_scales [num_blocks, kv_heads, block_size, 4 ceil(head_dim / 128)] uint8, v_scales
    [num_blocks, kv_heads, block_size] float32).  ``include/spec_kv.h`` says what
    they hold."""
    if head_dim % 32 or not 32 <= head_dim <= MAX_HEAD_DIM:
        raise ValueError(f"head_dim must be a multiple of 32 up to {MAX_HEAD_DIM}, got {head_dim}")
    rows = (num_blocks, kv_heads, block_size)

    def of(*last, dtype=torch.uint8):
        return torch.zeros((*rows, *last), dtype=dtype, device=device)
    return dict(k_codes=of(head_dim // 2), k_scales=of(-(-head_dim // 128) * 4),
                v_codes=of(head_dim // 2), v_scales=of(dtype=torch.float32))


def _cache_q4(cache, dev):
    """(blocks, kv_heads, block_size, head_dim) of a 4-bit cache on device ``dev``, and its
    pointers."""
    codes, u8 = cache["k_codes"], torch.uint8
    if codes.dim() != 4:
        raise ValueError("k_codes must be [num_blocks, kv_heads, block_size, head_dim / 2]")
    nb, kv, bs, half = shape = codes.shape
    if half % 16 or not 16 <= half <= MAX_HEAD_DIM // 2:
        raise ValueError(f"head_dim must be a multiple of 32 up to {MAX_HEAD_DIM}, got {2 * half}")
    return (nb, kv, bs, half * 2,
            (_tensor(codes, "k_codes", u8, shape, dev),
             _tensor(cache["k_scales"], "k_scales", u8, (nb, kv, bs, -(-half // 64) * 4), dev),
             _tensor(cache["v_codes"], "v_codes", u8, shape, dev),
             _tensor(cache["v_scales"], "v_scales", torch.float32, (nb, kv, bs), dev)))


def kv_cache_append_q4(k, v, slot_map, cache, *, q=None, positions=None, cos_sin=None,
                       interleaved=False, out=None):
    """Writes the rows of ``k`` and ``v`` [T, kv_heads, head_dim] (float32, bfloat16 or
    float16, parts of wider rows allowed) to their slots of a 4-bit ``cache``
    (``make_kv_cache_q4``) in place, rounded to its levels; skipped and differing slots
    as for ``kv_cache_append``.  With ``positions`` and ``cos_sin`` the keys, and ``q`` if
    there is one, are turned on the way as by ``kv_cache_append_rotary``, and the
    turned queries are returned (``out`` or a new tensor)."""
    lib = _pkg.library()
    dev = _gpu(k)
    nb, kv, bs, dim, pointers = _cache_q4(cache, dev)
    desc = _row_desc(k, v, kv, bs, nb, dim, dev)
    pq = pp = pc = po = None
    if cos_sin is not None:
        if positions is None:
            raise ValueError("cos_sin needs positions")
        pq, pp, pc, po, out = _rotation(desc, q, positions, cos_sin, interleaved, out, dev)
    elif q is not None or positions is not None or out is not None:
        raise ValueError("q, positions and out need cos_sin")
    _call(lib.kv_cache_append_q4, dev, ctypes.byref(desc), pq, k.data_ptr(), v.data_ptr(), pp, pc,
          _tensor(slot_map, "slot_map", torch.int64, (desc.tokens,), dev), po, *pointers)
    return out


def kv_cache_read_q4(slot_map, cache, dtype=torch.bfloat16):
    """The rows of the slots ``slot_map`` [T] int64 as they stand in a 4-bit ``cache``:
    (k, v), both [T, kv_heads, head_dim] of ``dtype``; 0 for slots that are negative or
    past the cache."""
    lib = _pkg.library()
    dev = _gpu(slot_map)
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    nb, kv, bs, dim, pointers = _cache_q4(cache, dev)
    if slot_map.dim() != 1:
        raise ValueError("slot_map must be [T]")
    T = _i32(slot_map.shape[0], "T")
    k, v = (torch.empty((T, kv, dim), dtype=dtype, device=slot_map.device) for _ in range(2))
    _call(lib.kv_cache_read_q4, dev, T, kv, dim, bs, _i32(nb, "num_blocks"), code,
          _tensor(slot_map, "slot_map", torch.int64, (T,), dev), *pointers, k.data_ptr(),
          v.data_ptr())
    return k, v


def _attention_q4_desc(q, cache, block_table, scale, sliding_window, max_new):
    code = _CODES.get(q.dtype)
    if code is None or code == 0:
        raise TypeError(f"q must be bfloat16 or float16, got {q.dtype}")
    nb, kv, bs, dim, pointers = _cache_q4(cache, q.get_device())
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
                         int(max_new), 0, stride, 0,
                         dim ** -0.5 if scale is None else float(scale), 0.0), pointers


def kv_paged_attention_q4_workspace_bytes(q, cache, block_table, *, sliding_window=0, max_new=0):
    """Workspace bytes of ``kv_paged_attention_q4`` on tensors of these shapes."""
    desc, _ = _attention_q4_desc(q, cache, block_table, None, sliding_window, max_new)
    return int(_pkg.library().kv_paged_attention_q4_workspace_bytes(ctypes.byref(desc)))


def kv_paged_attention_q4(q, cache, block_table, seq_lens, cu_tokens, *, scale=None,
                          sliding_window=0, max_new=0, lse=False, out=None, workspace=None):
    """``kv_paged_attention`` over a 4-bit ``cache``: ``q`` [T, heads, head_dim] bfloat16
    or float16, head_dim a multiple of 32 up to 256, everything else as there.  A query
    row that holds an infinity or NaN gives NaN; a value row that does makes ``out`` NaN
    where it is seen, and leaves ``lse``."""
    lib = _pkg.library()
    desc, pointers = _attention_q4_desc(q, cache, block_table, scale, sliding_window, max_new)
    return _attend(lib.kv_paged_attention_q4, lib.kv_paged_attention_q4_workspace_bytes, desc, q,
                   pointers, block_table, seq_lens, cu_tokens, lse, out, workspace)
