"""include/spec_kv.h on the CPU: exported symbols, workspace sizes and every
refusal of the paged-KV calls (host checks return before any HIP call), and the
checks of the Python binding."""

import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(0x1000)


@pytest.fixture(scope="module")
def sv():
    import lossless_token_verification_amd as m
    if not os.path.exists(m.LIB_PATH):
        from lossless_token_verification_amd import build
        build.build()
    m.library()
    return m


@pytest.fixture(scope="module")
def kv(sv):
    from lossless_token_verification_amd import kv as m
    return m


def test_every_declared_symbol_is_exported(sv):
    text = open(os.path.join(ROOT, "include", "spec_kv.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*(?:const\s+)?\w+\s*\**\s+\**(\w+)\s*\(", text, flags=re.M)
    assert sorted(names) == sorted(sv.KV_EXPORTED)
    lib = ctypes.CDLL(sv.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    assert sv.library().spec_kv_abi_version() == 1


EXTEND = dict(batch=2, max_blocks=4, block_size=16, table=P, lens=P, new=P, free=P, capacity=8,
              count=P, freed=None, max_freed=0, num_freed=None, max_tokens=4, new_lens=P, taken=P,
              left=P, cu=P, slots=P, positions=P)


def _extend(sv, **kw):
    a = {**EXTEND, **kw}
    return sv.library().kv_blocktable_extend(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(max_blocks=-1), 1), (dict(block_size=0), 1),
    (dict(capacity=-1), 1), (dict(max_freed=-1), 1), (dict(max_tokens=-1), 1),
    (dict(table=None), 1), (dict(lens=None), 1), (dict(new=None), 1), (dict(free=None), 1),
    (dict(count=None), 1), (dict(freed=P, max_freed=1), 1), (dict(new_lens=None), 1),
    (dict(taken=None), 1), (dict(left=None), 1), (dict(cu=None), 1), (dict(slots=None), 1),
    (dict(batch=(1 << 24) + 1), 2), (dict(max_tokens=(1 << 30) + 1), 2),
    (dict(table=ctypes.c_void_p(0x1002)), 3), (dict(slots=ctypes.c_void_p(0x1004)), 3),
    (dict(positions=ctypes.c_void_p(0x1001)), 3)])
def test_extend_refusals(sv, kw, status):
    assert _extend(sv, **kw) == status
    assert sv.library().spec_verify_last_error()


def _append(sv, kv, ptrs=None, **kw):
    d = dict(tokens=3, kv_heads=2, head_dim=64, block_size=16, num_blocks=4, dtype=1, k_stride=0,
             v_stride=0, block_stride=0)
    d.update(kw)
    p = dict(k=P, v=P, slots=P, kc=P, vc=P)
    p.update(ptrs or {})
    return sv.library().kv_cache_append(ctypes.byref(kv.AppendDesc(*d.values())), *p.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), 1), (dict(kv_heads=0), 1), (dict(kv_heads=1 << 17), 2),
    (dict(head_dim=0), 1), (dict(head_dim=5000), 2), (dict(block_size=0), 1),
    (dict(num_blocks=-1), 1), (dict(num_blocks=1 << 28, block_size=16), 2), (dict(dtype=3), 2),
    (dict(k_stride=127), 1), (dict(v_stride=1), 1), (dict(k_stride=2 ** 41), 1),
    (dict(block_stride=2047), 1), (dict(block_stride=2 ** 62), 1),
    (dict(ptrs=dict(k=None)), 1), (dict(ptrs=dict(slots=None)), 1),
    (dict(ptrs=dict(vc=None)), 1), (dict(ptrs=dict(k=ctypes.c_void_p(0x1001))), 3),
    (dict(ptrs=dict(slots=ctypes.c_void_p(0x1004))), 3)])
def test_append_refusals(sv, kv, kw, status):
    assert _append(sv, kv, **kw) == status
    assert sv.library().spec_verify_last_error()


def test_append_of_nothing(sv, kv):
    assert _append(sv, kv, tokens=0, ptrs=dict(k=None, v=None, slots=None)) == 0
    assert _append(sv, kv, num_blocks=0, ptrs=dict(kc=None, vc=None)) == 0
    assert sv.library().kv_cache_append(None, P, P, P, P, P, None) == 1


ATTEND = dict(batch=2, tokens=5, heads=8, kv_heads=2, head_dim=64, block_size=16, num_blocks=9,
              max_blocks=4, dtype=1, sliding_window=0, max_new=0, reserved=0, q_stride=0,
              block_stride=0, scale=0.125, reserved_f=0.0)


def _attend(sv, kv, ptrs=None, ws_bytes=1 << 40, **kw):
    d = {**ATTEND, **kw}
    p = dict(q=P, k=P, v=P, table=P, lens=P, cu=P, out=P, lse=None, ws=P)
    p.update(ptrs or {})
    return sv.library().kv_paged_attention(ctypes.byref(kv.AttentionDesc(*d.values())),
                                           *p.values(), ws_bytes, None)


def _ws(sv, kv, **kw):
    d = {**ATTEND, **kw}
    return sv.library().kv_paged_attention_workspace_bytes(
        ctypes.byref(kv.AttentionDesc(*d.values())))


BAD = [(dict(batch=-1), 1), (dict(batch=(1 << 24) + 1), 2), (dict(tokens=-1), 1), (dict(heads=0), 1), (dict(heads=7), 1),
       (dict(heads=1 << 17, kv_heads=1), 2), (dict(kv_heads=0), 1), (dict(head_dim=60), 2),
       (dict(head_dim=264), 2), (dict(head_dim=0), 1), (dict(block_size=0), 1),
       (dict(num_blocks=-1), 1), (dict(num_blocks=1 << 30), 2), (dict(max_blocks=-1), 1),
       (dict(dtype=3), 2), (dict(dtype=-1), 2), (dict(sliding_window=-1), 1),
       (dict(max_new=-1), 1), (dict(reserved=1), 1), (dict(reserved_f=1.0), 1),
       (dict(q_stride=511), 1), (dict(q_stride=516), 3), (dict(block_stride=2047), 1),
       (dict(block_stride=2052), 3), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
       (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
       (dict(scale=3e38), 1), (dict(tokens=2 ** 31 - 1), 2),
       (dict(tokens=2 ** 27, heads=8, kv_heads=8, dtype=0), 2)]


@pytest.mark.parametrize("kw,status", BAD)
def test_attention_refuses_descriptors(sv, kv, kw, status):
    assert _attend(sv, kv, **kw) == status
    assert sv.library().spec_verify_last_error()
    assert _ws(sv, kv, **kw) == 0


@pytest.mark.parametrize("ptrs,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(table=None), 1),
    (dict(lens=None), 1), (dict(cu=None), 1), (dict(out=None), 1),
    (dict(q=ctypes.c_void_p(0x1008)), 3), (dict(k=ctypes.c_void_p(0x1008)), 3),
    (dict(out=ctypes.c_void_p(0x1008)), 3), (dict(lse=ctypes.c_void_p(0x1002)), 3)])
def test_attention_refuses_pointers(sv, kv, ptrs, status):
    assert _attend(sv, kv, ptrs) == status


def test_attention_workspace(sv, kv):
    long = dict(max_blocks=4096, num_blocks=8192)
    need = _ws(sv, kv, **long)
    assert need > 0
    assert _attend(sv, kv, dict(ws=None), **long) == 4
    assert _attend(sv, kv, dict(ws=ctypes.c_void_p(0x1010)), **long) == 4
    assert _attend(sv, kv, ws_bytes=need - 1, **long) == 4
    # contexts of one split, and a window that keeps them so, need none
    assert _ws(sv, kv, max_blocks=4) == 0
    assert _ws(sv, kv, sliding_window=16, **long) == 0
    # nothing to do: no launch, no pointers
    for kw in (dict(batch=0), dict(tokens=0)):
        assert _attend(sv, kv, dict(q=None, k=None, v=None, table=None, lens=None, cu=None,
                                    out=None), **kw) == 0
    # extreme but valid descriptors stay within bounds
    for kw in (dict(tokens=2 ** 27, heads=8, kv_heads=8), dict(batch=2 ** 31 - 1, tokens=3),
               dict(max_blocks=2 ** 31 - 1, block_size=1 << 20, num_blocks=1),
               dict(sliding_window=2 ** 31 - 1, max_blocks=2 ** 31 - 1),
               dict(heads=1 << 16, kv_heads=1 << 16, max_blocks=2 ** 31 - 1)):
        _ws(sv, kv, **kw)


def _cpu_tensors(dtype=torch.bfloat16):
    return dict(q=torch.zeros((3, 4, 64), dtype=dtype),
                k_cache=torch.zeros((5, 2, 16, 64), dtype=dtype),
                v_cache=torch.zeros((5, 2, 16, 64), dtype=dtype),
                block_table=torch.zeros((2, 3), dtype=torch.int32),
                seq_lens=torch.zeros(2, dtype=torch.int32),
                cu_tokens=torch.zeros(3, dtype=torch.int32))


@pytest.mark.parametrize("change,error", [
    (dict(q=torch.zeros((3, 4, 64), dtype=torch.float64)), TypeError),
    (dict(q=torch.zeros((3, 4, 32), dtype=torch.bfloat16)), ValueError),
    (dict(q=torch.zeros((3, 64, 4), dtype=torch.bfloat16).transpose(1, 2)), ValueError),
    (dict(k_cache=torch.zeros((5, 2, 16, 64))), ValueError),
    (dict(k_cache=torch.zeros((5, 16, 2, 64), dtype=torch.bfloat16).transpose(1, 2)), ValueError),
    (dict(v_cache=torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)), ValueError),
    (dict(v_cache=torch.zeros((5, 2, 2, 16, 64), dtype=torch.bfloat16)[:, 0]), ValueError),
    (dict(block_table=torch.zeros((2, 3), dtype=torch.int64)), ValueError),
    (dict(seq_lens=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(cu_tokens=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(), ValueError)])   # host tensors are no device tensors
def test_binding_refusals_attention(sv, change, error):
    with pytest.raises(error):
        sv.kv_paged_attention(**{**_cpu_tensors(), **change})


def test_binding_refusals_others(sv):
    i = torch.zeros(2, dtype=torch.int32)
    table, free, one = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(9, dtype=torch.int32), \
        torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):      # host tensors
        sv.kv_blocktable_extend(table, i, i, free, one, 16, 4)
    with pytest.raises(ValueError):
        sv.kv_blocktable_extend(table, i.long(), i, free, one, 16, 4)
    with pytest.raises(ValueError):
        sv.kv_blocktable_extend(table, i, i, free, one, 16, -1)
    with pytest.raises(ValueError):
        sv.kv_blocktable_extend(table, i, i, free, one, 16, 4, freed_blocks=table)
    with pytest.raises(ValueError):
        sv.kv_blocktable_extend(table, i, i, free, one, 16, 2 ** 32 + 4)
    with pytest.raises(ValueError):
        sv.kv_blocktable_extend(table, i, i, free, one, 2 ** 32 + 16, 4)
    c = torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    for args in ((k, k, slots, c, c),                                    # host tensors
                 (k[:2], k, slots, c, c), (k, k, slots[:2], c, c), (k, k.float(), slots, c, c),
                 (k, k, slots.int(), c, c), (k, k, slots, c, c.transpose(1, 2))):
        with pytest.raises(ValueError):
            sv.kv_cache_append(*args)
    with pytest.raises(TypeError):
        sv.kv_cache_append(k.double(), k.double(), slots, c, c)


def test_binding_refuses_overlapping_rows_and_blocks(sv):
    t = _cpu_tensors()
    row = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="rows must not overlap"):
        sv.kv_paged_attention(**{**t, "q": row.expand(3, 4, 64)})
    wide = torch.zeros((1, 2, 16, 64), dtype=torch.bfloat16).expand(5, 2, 16, 64)
    with pytest.raises(ValueError, match="blocks of a cache"):
        sv.kv_paged_attention(**{**t, "k_cache": wide, "v_cache": wide})
    with pytest.raises(ValueError, match="rows must not overlap"):
        sv.kv._row_stride(row.expand(3, 4, 64), "k")
    # one row has no stride to speak of
    assert sv.kv._row_stride(row, "k") == 0
    assert sv.kv._caches(wide[:1], wide[:1], torch.bfloat16, -1)[4] == 0


@pytest.mark.parametrize("name", ["sliding_window", "max_new"])
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32 + 4, -2 ** 32 + 1])
def test_binding_refuses_numbers_beyond_32_bits(sv, name, value):
    with pytest.raises(ValueError, match="32-bit"):
        sv.kv_paged_attention(**_cpu_tensors(), **{name: value})
