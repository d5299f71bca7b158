"""GPU tests of kv_cache_append_q4 and kv_cache_read_q4 against the oracle: codes and
units of every row, bit for bit."""

import math

import numpy as np
import pytest
import torch

from oracle import kvq4
from tests import kvcases as C
from tests import kvq4cases as Q
from tests.test_gpu_kv_rotary import rows_case, table, turned_bound

pytestmark = pytest.mark.gpu

DEV = C.DEV


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_token_verification_amd as m
    m.library()
    return m


def _cache(sv, blocks, kv, bs, dim, seed=0):
    """A cache full of other bytes."""
    cache = sv.make_kv_cache_q4(blocks, kv, bs, dim, DEV)
    g = torch.Generator().manual_seed(seed)
    for n in ("k_codes", "v_codes", "k_scales"):
        cache[n].copy_(torch.randint(0, 256, cache[n].shape, generator=g, dtype=torch.uint8))
    cache["v_scales"].fill_(77.0)
    return cache


def _check_rows(cache, before, k, v, slots, held, dim, bs):
    """The rows at the held slots are the float32 rows k, v coded by the oracle;
    everything else is as before."""
    c = {n: t.cpu().numpy() for n, t in cache.items()}
    for t in np.nonzero(held)[0]:
        page, at = int(slots[t]) // bs, int(slots[t]) % bs
        for h in range(k.shape[1]):
            codes, units = kvq4.code_keys(k[t, h])
            got = c["k_codes"][page, h, at]
            got = np.stack([got & 15, got >> 4], -1).reshape(-1)
            fine = np.repeat(np.array(units) != 255, 32)
            assert np.array_equal(got[fine], np.array(codes)[fine]), (t, h)
            assert c["k_scales"][page, h, at, :dim // 32].tolist() == units, (t, h)
            codes, unit = kvq4.code_values(v[t, h])
            got = c["v_codes"][page, h, at]
            got = np.stack([got & 15, got >> 4], -1).reshape(-1)
            assert np.array_equal(c["v_scales"][page, h, at], unit, equal_nan=True), (t, h)
            if unit > 0:
                assert got.tolist() == codes, (t, h)
    mask = np.ones(c["v_scales"].shape, dtype=bool)
    for t in np.nonzero(held)[0]:
        mask[int(slots[t]) // bs, :, int(slots[t]) % bs] = False
    for n in Q.CACHE:
        assert np.array_equal(c[n][mask], before[n].cpu().numpy()[mask]), n


CASES = [
    # (T, heads, kv, dim, rot, pairs, block size, dtype, fused)
    (1, 32, 8, 128, 0, False, 16, "bf16", True),
    (37, 2, 1, 64, 0, False, 1, "f32", False),
    (60, 0, 5, 96, 0, False, 24, "f16", True),
    (65, 6, 3, 32, 0, False, 7, "bf16", True),
    (40, 8, 2, 256, 0, False, 64, "f16", False),
    (1, 32, 8, 128, 128, False, 16, "bf16", True),
    (50, 2, 2, 64, 64, True, 16, "f16", False),
    (30, 3, 1, 160, 100, False, 9, "bf16", True),     # half the turned part: no whole vectors
    (30, 3, 1, 224, 96, False, 9, "f32", False),
    (33, 4, 2, 96, 96, False, 16, "f16", True),       # groups that straddle the halves
    (20, 4, 4, 256, 200, True, 16, "bf16", False),
    (31, 0, 2, 32, 32, True, 4, "f32", True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"T{c[0]}h{c[1]}-{c[2]}d{c[3]}r{c[4]}"
                         f"{'p' if c[5] else 'h'}{c[7]}")
def test_append_parity(sv, case):
    T, heads, kv, dim, rot, pairs, bs, dt, fused = case
    c = rows_case(T, heads, kv, dim, bs, dt, fused, T + dim)
    wide = c["k"]._base.to(DEV)
    part = {n: wide.as_strided(c[n].size(), c[n].stride(), c[n].storage_offset()) for n in "qkv"}
    cache = _cache(sv, c["blocks"], kv, bs, dim)
    before = {n: t.clone() for n, t in cache.items()}
    pos = c["positions"].tolist()
    known = np.array([0 <= p < 500 for p in pos]) if rot else np.ones(T, dtype=bool)
    held = known & np.array([0 <= s < c["blocks"] * bs for s in c["slots"].tolist()])
    turn = {}
    if rot:
        cs = table(500, rot)
        turn = dict(positions=c["positions"].to(DEV), cos_sin=cs.to(DEV), interleaved=pairs)
        if heads:
            turn.update(q=part["q"], out=torch.full((T, heads, dim), 7.0, dtype=C.DT[dt], device=DEV))
    r = sv.kv_cache_append_q4(part["k"], part["v"], c["slots"].to(DEV), cache, **turn)
    torch.cuda.synchronize()
    k = C.to64(c["k"])
    if rot:
        k = kvq4.rotate(k, pos, cs.numpy(), pairs)
    _check_rows(cache, before, k.astype(np.float32), C.to64(c["v"]).astype(np.float32), c["slots"],
                held, dim, bs)
    if rot and heads:
        ref = kvq4.rotate(C.to64(c["q"]), pos, cs.numpy(), pairs)
        bound = turned_bound(C.to64(c["q"]), cs.numpy(), pos, pairs, dt)
        assert (np.abs(C.to64(r) - ref)[known] <= bound[known]).all()
        assert (C.to64(r)[~known] == 7.0).all()
    else:
        assert r is None
    # the rows read back are what the codes stand for
    for out in ("f32", "bf16", "f16"):
        rk, rv = sv.kv_cache_read_q4(c["slots"].to(DEV), cache, C.DT[out])
        torch.cuda.synchronize()
        assert rk.shape == (T, kv, dim) and rk.dtype is C.DT[out]
        n = {n: t.cpu().numpy() for n, t in cache.items()}
        for t, s in enumerate(c["slots"].tolist()):
            if not 0 <= s < c["blocks"] * bs:
                assert (rk[t] == 0).all() and (rv[t] == 0).all()
                continue
            at = (s // bs, slice(None), s % bs)
            if not held[t]:
                continue
            want = torch.from_numpy(kvq4.key_values(n["k_codes"][at], n["k_scales"][at]))
            assert torch.equal(rk[t].cpu(), want.to(C.DT[out])), (t, out)
            want = torch.from_numpy(kvq4.value_values(n["v_codes"][at], n["v_scales"][at]))
            assert torch.equal(rv[t].cpu(), want.float().to(C.DT[out])), (t, out)


def test_every_border_and_size(sv):
    """Rows of borders between levels, at units over the whole range, and of what is
    not finite."""
    dim, levels = 64, torch.tensor(kvq4.MAGNITUDES)
    mid = (levels[1:] + levels[:-1]) / 2
    base = torch.cat([levels, mid, torch.tensor([6.5, 7.0])])
    near = torch.cat([base, torch.nextafter(base, torch.tensor(-9.0)),
                      torch.nextafter(base, torch.tensor(9.0))])
    near = torch.cat([near, -near])
    rows = []
    for e in (-149, -140, -127, -126, -125, -30, 0, 1, 60, 120, 124, 125):
        for i in range(0, len(near), dim - 2):
            part = near[i:i + dim - 2]
            for top in (6.0, 7.0, 4.0):
                row = torch.zeros(dim)
                row[:len(part)] = part
                row[30], row[62] = top, top          # the unit of either half, and of a value row
                rows.append(torch.ldexp(row, torch.tensor(e)))
    for bad in (math.inf, -math.inf, math.nan):
        row = torch.ones(dim)
        row[40] = bad
        rows.append(row)
    rows = torch.stack(rows)[:, None]
    T = len(rows)
    for dt in ("f32", "bf16", "f16"):
        x = rows.to(C.DT[dt])
        cache = _cache(sv, -(-T // 16), 1, 16, dim)
        before = {n: t.clone() for n, t in cache.items()}
        slots = torch.randperm(-(-T // 16) * 16, generator=torch.Generator().manual_seed(1))[:T]
        sv.kv_cache_append_q4(x.to(DEV), x.to(DEV), slots.to(DEV), cache)
        torch.cuda.synchronize()
        f = x.float().numpy()
        _check_rows(cache, before, f, f, slots, np.ones(T, dtype=bool), dim, 16)
        rk, rv = sv.kv_cache_read_q4(slots.to(DEV), cache, torch.float32)
        torch.cuda.synchronize()
        bad = ~torch.isfinite(x[:, 0].float()).all(-1)
        assert torch.isnan(rv.cpu()[bad]).all() and not torch.isnan(rv.cpu()[~bad]).any()
        assert not torch.isnan(rk.cpu()[~bad]).any()


def test_rows_off_16_bytes(sv):
    for rot, pairs in ((0, False), (64, False), (64, True)):
        c = rows_case(45, 4, 2, 64, 16, "bf16", False, 5, extra=1)
        cs = table(500, 64).to(DEV)
        wide = c["k"]._base.to(DEV)
        q, k, v = (wide.as_strided(c[n].size(), c[n].stride(), c[n].storage_offset()) for n in "qkv")
        a, b = _cache(sv, c["blocks"], 2, 16, 64), _cache(sv, c["blocks"], 2, 16, 64)
        turn = dict(positions=c["positions"].to(DEV), cos_sin=cs, interleaved=pairs) if rot else {}
        more = lambda x: dict(turn, q=x, out=torch.zeros_like(q.contiguous())) if rot else {}  # noqa: E731
        slots = c["slots"].to(DEV)
        ra = sv.kv_cache_append_q4(k, v, slots, a, **more(q))
        rb = sv.kv_cache_append_q4(k.contiguous(), v.contiguous(), slots, b, **more(q.contiguous()))
        torch.cuda.synchronize()
        assert ra is None and rb is None or torch.equal(ra, rb)
        for n in Q.CACHE:
            assert torch.equal(a[n], b[n]), n


def test_empty_calls_and_no_blocks(sv):
    cs = table(10, 64).to(DEV)
    e = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    z = torch.zeros(0, dtype=torch.int64, device=DEV)
    cache = sv.make_kv_cache_q4(3, 2, 16, 64, DEV)
    sv.kv_cache_append_q4(e, e, z, cache)
    assert sv.kv_cache_read_q4(z, cache)[0].shape == (0, 2, 64)
    none = sv.make_kv_cache_q4(0, 2, 16, 64, DEV)
    x = torch.randn((3, 2, 64), device=DEV).bfloat16()
    pos = torch.tensor([0, 5, 9], dtype=torch.int32, device=DEV)
    slots = torch.arange(3, device=DEV)
    sv.kv_cache_append_q4(x, x, slots, none)
    r = sv.kv_cache_append_q4(x, x, slots, none, q=x, positions=pos, cos_sin=cs)
    full = sv.kv_cache_append_q4(x, x, slots, cache, q=x, positions=pos, cos_sin=cs)
    k, v = sv.kv_cache_read_q4(slots, none)
    torch.cuda.synchronize()
    assert torch.equal(r, full) and (k == 0).all() and (v == 0).all()


def test_slots_beyond_32_bits_of_bytes(sv):
    """A cache whose codes take more than 2^32 bytes."""
    nb, kv, bs, dim = 2 ** 17 + 8, 4, 64, 256
    cache = dict(k_codes=torch.zeros((nb, kv, bs, dim // 2), dtype=torch.uint8, device=DEV),
                 v_codes=torch.zeros((nb, kv, bs, dim // 2), dtype=torch.uint8, device=DEV),
                 k_scales=torch.zeros((nb, kv, bs, 8), dtype=torch.uint8, device=DEV),
                 v_scales=torch.zeros((nb, kv, bs), dtype=torch.float32, device=DEV))
    assert cache["k_codes"].numel() > 2 ** 32
    small = sv.make_kv_cache_q4(8, kv, bs, dim, DEV)
    x = torch.randn((20, kv, dim), device=DEV).half()
    y = torch.randn((20, kv, dim), device=DEV).half()
    slots = torch.randperm(8 * bs, device=DEV)[:20]
    sv.kv_cache_append_q4(x, y, slots, small)
    sv.kv_cache_append_q4(x, y, slots + 2 ** 17 * bs, cache)
    torch.cuda.synchronize()
    for n in Q.CACHE:
        assert torch.equal(cache[n][2 ** 17:], small[n]), n
    a, b = sv.kv_cache_read_q4(slots + 2 ** 17 * bs, cache), sv.kv_cache_read_q4(slots, small)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert not cache["k_codes"][:2 ** 17].any()
