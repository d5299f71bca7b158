"""The rotated append and the calls of the 4-bit cache on the CPU: every refusal
(host checks return before any HIP call), workspace sizes, and the checks of the
Python binding."""

import ctypes

import pytest
import torch

from tests.test_kv_abi_cpu import P, kv, sv   # noqa: F401

ODD = {n: ctypes.c_void_p(0x1000 + n) for n in (1, 2, 4, 8)}

ROWS = dict(tokens=3, heads=4, kv_heads=2, head_dim=64, block_size=16, num_blocks=4, dtype=1,
            rotary_dim=64, interleaved=0, table_rows=100, q_stride=0, k_stride=0, v_stride=0,
            q_out_stride=0, block_stride=0)
ROW_PTRS = dict(q=P, k=P, v=P, positions=P, cos_sin=P, slots=P, q_out=P)


def _rotary(sv, kv, ptrs=None, **kw):   # noqa: F811
    p = dict(ROW_PTRS, k_cache=P, v_cache=P)
    p.update(ptrs or {})
    d = kv.RotaryDesc(*{**ROWS, **kw}.values())
    return sv.library().kv_cache_append_rotary(ctypes.byref(d), *p.values(), None)


def _store(sv, kv, ptrs=None, **kw):   # noqa: F811
    p = dict(ROW_PTRS, k_codes=P, k_scales=P, v_codes=P, v_scales=P)
    p.update(ptrs or {})
    d = kv.RotaryDesc(*{**ROWS, **kw}.values())
    return sv.library().kv_cache_append_q4(ctypes.byref(d), *p.values(), None)


BOTH = [(dict(tokens=-1), 1), (dict(heads=-1), 1), (dict(heads=1 << 17), 2), (dict(kv_heads=0), 1),
        (dict(kv_heads=1 << 17), 2), (dict(head_dim=0), 1), (dict(head_dim=8192), 2),
        (dict(block_size=0), 1), (dict(num_blocks=-1), 1), (dict(num_blocks=1 << 28), 2),
        (dict(dtype=3), 2), (dict(rotary_dim=-2), 1), (dict(rotary_dim=66), 1),
        (dict(rotary_dim=7), 1), (dict(rotary_dim=0), 1), (dict(interleaved=2), 1),
        (dict(interleaved=-1), 1), (dict(table_rows=-1), 1), (dict(q_stride=255), 1),
        (dict(k_stride=127), 1), (dict(v_stride=1), 1), (dict(q_out_stride=2 ** 41), 1),
        (dict(q_stride=-1), 1),
        (dict(ptrs=dict(q=None)), 1), (dict(ptrs=dict(k=None)), 1), (dict(ptrs=dict(v=None)), 1),
        (dict(ptrs=dict(positions=None)), 1), (dict(ptrs=dict(cos_sin=None)), 1),
        (dict(ptrs=dict(slots=None)), 1), (dict(ptrs=dict(q_out=None)), 1),
        (dict(ptrs=dict(q=ODD[1])), 3), (dict(ptrs=dict(v=ODD[1])), 3),
        (dict(ptrs=dict(positions=ODD[2])), 3), (dict(ptrs=dict(cos_sin=ODD[2])), 3),
        (dict(ptrs=dict(slots=ODD[4])), 3)]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(block_stride=2047), 1), (dict(block_stride=2 ** 62), 1),
    (dict(ptrs=dict(k_cache=None)), 1), (dict(ptrs=dict(v_cache=ODD[1])), 3)])
def test_rotary_append_refusals(sv, kv, kw, status):   # noqa: F811
    assert _rotary(sv, kv, **kw) == status
    assert sv.library().spec_verify_last_error()


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(head_dim=48, rotary_dim=48), 2), (dict(head_dim=288), 2), (dict(block_stride=2048), 1),
    (dict(rotary_dim=0, heads=1), 1), (dict(ptrs=dict(k_codes=None)), 1),
    (dict(ptrs=dict(v_scales=None)), 1), (dict(ptrs=dict(k_codes=ODD[8])), 3),
    (dict(ptrs=dict(v_codes=ODD[4])), 3), (dict(ptrs=dict(k_scales=ODD[2])), 3),
    (dict(ptrs=dict(v_scales=ODD[1])), 3)])
def test_q4_append_refusals(sv, kv, kw, status):   # noqa: F811
    assert _store(sv, kv, **kw) == status
    assert sv.library().spec_verify_last_error()


def test_appends_of_nothing(sv, kv):   # noqa: F811
    none = dict.fromkeys(ROW_PTRS)
    assert _rotary(sv, kv, none, tokens=0) == 0
    assert _rotary(sv, kv, dict(none, k_cache=None, v_cache=None), tokens=0, num_blocks=0) == 0
    assert _store(sv, kv, none, tokens=0) == 0
    # rows without a cache and without queries
    assert _rotary(sv, kv, dict(k_cache=None, v_cache=None), heads=0, num_blocks=0) == 0
    assert _store(sv, kv, dict(k_codes=None, k_scales=None, v_codes=None, v_scales=None), heads=0,
                  num_blocks=0) == 0
    lib = sv.library()
    assert lib.kv_cache_append_rotary(None, *[P] * 9, None) == 1
    assert lib.kv_cache_append_q4(None, *[P] * 11, None) == 1


READ = dict(tokens=3, kv_heads=2, head_dim=64, block_size=16, num_blocks=4, dtype=1)
READ_PTRS = dict(slots=P, k_codes=P, k_scales=P, v_codes=P, v_scales=P, k=P, v=P)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), 1), (dict(kv_heads=0), 1), (dict(head_dim=0), 1), (dict(head_dim=40), 2),
    (dict(head_dim=288), 2), (dict(block_size=0), 1), (dict(num_blocks=-1), 1),
    (dict(num_blocks=1 << 28), 2), (dict(dtype=3), 2), (dict(ptrs=dict(slots=None)), 1),
    (dict(ptrs=dict(slots=ODD[4])), 3), (dict(ptrs=dict(k_codes=None)), 1),
    (dict(ptrs=dict(v_codes=ODD[8])), 3), (dict(ptrs=dict(k_scales=ODD[2])), 3),
    (dict(ptrs=dict(v_scales=None)), 1), (dict(ptrs=dict(k=None)), 1),
    (dict(ptrs=dict(k=ODD[8])), 3), (dict(ptrs=dict(v=ODD[8])), 3)])
def test_q4_read_refusals(sv, kw, status):   # noqa: F811
    kw = dict(kw)
    p = {**READ_PTRS, **kw.pop("ptrs", {})}
    assert sv.library().kv_cache_read_q4(*{**READ, **kw}.values(), *p.values(), None) == status
    assert sv.library().spec_verify_last_error()


def test_q4_read_of_nothing(sv):   # noqa: F811
    p = dict.fromkeys(READ_PTRS)
    assert sv.library().kv_cache_read_q4(*{**READ, "tokens": 0}.values(), *p.values(), None) == 0


ATTEND = dict(batch=2, tokens=5, heads=8, kv_heads=2, head_dim=64, block_size=16, num_blocks=9,
              max_blocks=4, dtype=1, sliding_window=0, max_new=0, reserved=0, q_stride=0,
              block_stride=0, scale=0.125, reserved_f=0.0)


def _attend(sv, kv, ptrs=None, ws_bytes=1 << 40, **kw):   # noqa: F811
    p = dict(q=P, k_codes=P, k_scales=P, v_codes=P, v_scales=P, table=P, lens=P, cu=P, out=P,
             lse=None, ws=P)
    p.update(ptrs or {})
    d = kv.AttentionDesc(*{**ATTEND, **kw}.values())
    return sv.library().kv_paged_attention_q4(ctypes.byref(d), *p.values(), ws_bytes, None)


def _ws(sv, kv, **kw):   # noqa: F811
    d = kv.AttentionDesc(*{**ATTEND, **kw}.values())
    return sv.library().kv_paged_attention_q4_workspace_bytes(ctypes.byref(d))


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(batch=(1 << 16) + 1), 2), (dict(tokens=-1), 1), (dict(heads=0), 1),
    (dict(heads=7), 1), (dict(heads=1 << 17, kv_heads=1), 2), (dict(kv_heads=0), 1),
    (dict(head_dim=0), 1), (dict(head_dim=72), 2), (dict(head_dim=288), 2),
    (dict(block_size=0), 1), (dict(num_blocks=-1), 1), (dict(num_blocks=1 << 30), 2),
    # rows of the cache are numbered in 32 bits
    (dict(num_blocks=1 << 26, heads=32, kv_heads=8), 2),
    (dict(max_blocks=-1), 1), (dict(dtype=0), 2), (dict(dtype=3), 2), (dict(sliding_window=-1), 1),
    (dict(max_new=-1), 1), (dict(reserved=1), 1), (dict(reserved_f=1.0), 1),
    (dict(q_stride=511), 1), (dict(q_stride=516), 3), (dict(block_stride=2048), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(scale=3e38), 1), (dict(tokens=2 ** 31 - 1), 2)])
def test_q4_attention_refuses_descriptors(sv, kv, kw, status):   # noqa: F811
    assert _attend(sv, kv, **kw) == status
    assert sv.library().spec_verify_last_error()
    assert _ws(sv, kv, **kw) == 0


@pytest.mark.parametrize("ptrs,status", [
    (dict(q=None), 1), (dict(k_codes=None), 1), (dict(k_scales=None), 1), (dict(v_codes=None), 1),
    (dict(v_scales=None), 1), (dict(table=None), 1), (dict(lens=None), 1), (dict(cu=None), 1),
    (dict(out=None), 1), (dict(q=ODD[8]), 3), (dict(k_codes=ODD[8]), 3), (dict(k_scales=ODD[2]), 3),
    (dict(v_codes=ODD[4]), 3), (dict(v_scales=ODD[1]), 3), (dict(out=ODD[8]), 3),
    (dict(lse=ODD[2]), 3)])
def test_q4_attention_refuses_pointers(sv, kv, ptrs, status):   # noqa: F811
    assert _attend(sv, kv, ptrs) == status


def test_q4_attention_workspace(sv, kv):   # noqa: F811
    long = dict(max_blocks=4096, num_blocks=8192)
    need = _ws(sv, kv, **long)
    assert need > 0
    assert _attend(sv, kv, dict(ws=None), **long) == 4
    assert _attend(sv, kv, dict(ws=ctypes.c_void_p(0x1010)), **long) == 4
    assert _attend(sv, kv, ws_bytes=need - 1, **long) == 4
    # contexts of one unit, and a window that keeps them so, need none
    assert _ws(sv, kv, max_blocks=8) == 0
    assert _ws(sv, kv, sliding_window=16, tokens=2, **long) < need
    for kw in (dict(batch=0), dict(tokens=0)):
        assert _attend(sv, kv, dict.fromkeys(("q", "k_codes", "k_scales", "v_codes", "v_scales", "table",
                                              "lens", "cu", "out")), **kw) == 0
    # the largest cache and batch that are taken (no q: refused for that alone)
    assert _attend(sv, kv, dict(q=None), num_blocks=(1 << 27) - 1, heads=16, kv_heads=2) == 1
    assert _attend(sv, kv, dict(q=None), batch=1 << 16, tokens=1 << 16) == 1
    assert b"q is NULL" in sv.library().spec_verify_last_error()


def _q4(nb=5, heads=2, bs=16, dim=64):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)   # noqa: E731
    return dict(k_codes=u8(nb, heads, bs, dim // 2), k_scales=u8(nb, heads, bs, -(-dim // 128) * 4),
                v_codes=u8(nb, heads, bs, dim // 2), v_scales=torch.zeros((nb, heads, bs)))


def _args():
    return dict(q=torch.zeros((3, 4, 64), dtype=torch.bfloat16), cache=_q4(),
                block_table=torch.zeros((2, 3), dtype=torch.int32),
                seq_lens=torch.zeros(2, dtype=torch.int32), cu_tokens=torch.zeros(3, dtype=torch.int32))


@pytest.mark.parametrize("change,error", [
    (dict(q=torch.zeros((3, 4, 64))), TypeError),
    (dict(q=torch.zeros((3, 4, 32), dtype=torch.bfloat16)), ValueError),
    (dict(q=torch.zeros((1, 4, 64), dtype=torch.bfloat16).expand(3, 4, 64)), ValueError),
    (dict(cache=_q4(dim=40)), ValueError), (dict(cache=_q4(dim=288)), ValueError),
    (dict(cache=dict(_q4(), v_codes=_q4(nb=4)["v_codes"])), ValueError),
    (dict(cache=dict(_q4(), k_scales=_q4(dim=256)["k_scales"])), ValueError),
    (dict(cache=dict(_q4(), v_scales=_q4()["v_scales"].bfloat16())), ValueError),
    (dict(cache=dict(_q4(), k_codes=_q4()["k_codes"].view(torch.int8))), ValueError),
    (dict(cache=dict(_q4(), k_codes=_q4()["k_codes"][0])), ValueError),
    (dict(block_table=torch.zeros((2, 3), dtype=torch.int64)), ValueError),
    (dict(seq_lens=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(sliding_window=2 ** 31), ValueError), (dict(max_new=2 ** 32 + 4), ValueError),
    (dict(), ValueError)])   # host tensors are no device tensors
def test_binding_refusals_attention(sv, change, error):   # noqa: F811
    with pytest.raises(error):
        sv.kv_paged_attention_q4(**{**_args(), **change})


def test_binding_refusals_rows(sv):   # noqa: F811
    k, slots = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    c = torch.zeros((5, 2, 16, 64), dtype=torch.bfloat16)
    q, pos, cs = torch.zeros((3, 4, 64), dtype=torch.bfloat16), slots.int(), torch.zeros((9, 64))
    with pytest.raises(ValueError, match="GPU"):
        sv.kv_cache_append_rotary(q, k, k, pos, cs, slots, c, c)
    with pytest.raises(ValueError, match="GPU"):
        sv.kv_cache_append_q4(k, k, slots, _q4())
    with pytest.raises(ValueError, match="GPU"):
        sv.kv_cache_read_q4(slots, _q4())
    # the shapes themselves, with the device out of the way
    row = sv.kv._row_desc
    with pytest.raises(TypeError):
        row(k.double(), k.double(), 2, 16, 5, 64, -1)
    for a, b in ((k, k[:2]), (k, k.float()), (k[:, :1], k[:, :1]), (k[:1].expand(3, 2, 64),) * 2):
        with pytest.raises(ValueError):
            row(a, b, 2, 16, 5, 64, -1)
    desc = row(k, k, 2, 16, 5, 64, -1)
    turn = sv.kv._rotation
    for bad in (dict(q=q[:2]), dict(q=q.float()), dict(q=q[..., :32]), dict(positions=pos.long()),
                dict(positions=pos[:2]), dict(cos_sin=cs.double()), dict(cos_sin=cs[0]),
                dict(cos_sin=cs[:, ::2]), dict(out=q[:2]), dict(out=q.float()),
                dict(q=None, out=q), dict(out=q[:1].expand(3, 4, 64))):
        a = dict(dict(q=q, positions=pos, cos_sin=cs, interleaved=False, out=None), **bad)
        with pytest.raises(ValueError):
            turn(desc, *a.values(), -1)
    assert turn(desc, q, pos, cs, True, q, -1)[4] is q
    for dim in (0, 16, 40, 288):
        with pytest.raises(ValueError, match="multiple of 32"):
            sv.make_kv_cache_q4(3, 2, 16, dim, device="cpu")
    made = sv.make_kv_cache_q4(3, 2, 16, 160, device="cpu")
    assert {n: t.shape for n, t in made.items()} == {n: t.shape for n, t in _q4(3, 2, 16, 160).items()}
