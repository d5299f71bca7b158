"""GPU parity of kv_cache_append_rotary with the float64 oracle."""

import numpy as np
import pytest
import torch

from oracle import kvq4
from tests import kvcases as C

pytestmark = pytest.mark.gpu

DEV = C.DEV


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_token_verification_amd as m
    m.library()
    return m


def table(rows, rot):
    """[rows, rot] cosines and sines, angles in float64."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def rows_case(T, heads, kv, dim, bs, dtype, fused, seed, extra=0, positions=500):
    """Rows of a projection, their slots (some of them none, each differing) and
    positions (some of them in no table), on the CPU."""
    g = torch.Generator().manual_seed(seed)
    dt = C.DT[dtype]
    lead = 8 if fused else 0
    wide = torch.randn((T, lead + (heads + 2 * kv) * dim + extra), generator=g).to(dt)
    nb = -(-2 * T // bs) + 2
    slots = torch.randperm(nb * bs, generator=g)[:T]
    odd = torch.tensor([-1, -2 ** 62, nb * bs, 2 ** 40, 2 ** 32 + 3])
    slots[::7] = odd[torch.arange(len(slots[::7])) % 5]
    pos = torch.randint(0, positions, (T,), generator=g, dtype=torch.int32)
    pos[3::11] = torch.tensor([-1, positions, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)[
        torch.arange(len(pos[3::11])) % 4]
    at = lambda i, n: wide[:, lead + i * dim:lead + (i + n) * dim].view(T, n, dim)  # noqa: E731
    return dict(q=at(0, heads), k=at(heads, kv), v=at(heads + kv, kv), slots=slots, positions=pos,
                blocks=nb)


def turned_bound(x, cs, pos, pairs, dtype):
    """Float32 products and their sum (a step and a half of the absolute sum), then
    half a step of the type."""
    size = kvq4.rotate(np.abs(x), pos, np.concatenate([np.abs(cs[:, :cs.shape[1] // 2]),
                                                       -np.abs(cs[:, cs.shape[1] // 2:])], 1), pairs)
    size2 = kvq4.rotate(np.abs(x), pos, np.abs(cs), pairs)
    size = np.maximum(np.abs(size), np.abs(size2))          # |x| |cos| + |y| |sin|
    half = torch.finfo(C.DT[dtype]).eps / 2
    tiny = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -149}[dtype]
    return (2.0 ** -23 + half) * 1.001 * size + tiny


CASES = [
    # (T, heads, kv, dim, rot, pairs, block size, dtype, fused)
    (1, 32, 8, 128, 128, False, 16, "bf16", True),
    (37, 2, 1, 64, 64, True, 1, "f16", False),
    (100, 15, 5, 80, 48, True, 24, "f16", True),
    (65, 6, 3, 40, 40, False, 7, "bf16", True),       # half a head is no whole vectors
    (300, 8, 8, 256, 64, False, 64, "f32", False),
    (29, 4, 2, 96, 96, False, 16, "bf16", False),
    (40, 3, 3, 5, 4, True, 3, "f32", True),           # no 16-byte rows
    (33, 7, 1, 9, 2, False, 5, "bf16", True),
    (50, 4, 2, 64, 2, True, 16, "f32", False),
    (2304, 32, 8, 128, 128, False, 16, "bf16", True),
    (129, 0, 2, 128, 128, True, 16, "f16", True),     # keys alone
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"T{c[0]}h{c[1]}-{c[2]}d{c[3]}r{c[4]}"
                         f"{'p' if c[5] else 'h'}{c[7]}")
def test_rotary_append_parity(sv, case):
    T, heads, kv, dim, rot, pairs, bs, dt, fused = case
    c = rows_case(T, heads, kv, dim, bs, dt, fused, T)
    cs = table(500, rot)
    g = torch.Generator().manual_seed(1)
    both = torch.randn((c["blocks"], 2, kv, bs, dim), generator=g).to(C.DT[dt])
    wide = c["k"]._base.to(DEV)
    part = {n: wide.as_strided(c[n].size(), c[n].stride(), c[n].storage_offset())
            for n in ("q", "k", "v")}
    dev = both.to(DEV)
    caches = (dev[:, 0], dev[:, 1]) if fused else (dev[:, 0].contiguous(), dev[:, 1].contiguous())
    before = [x.clone() for x in caches]
    out = torch.full((T, heads, dim), 7.0, dtype=C.DT[dt], device=DEV) if heads else None
    r = sv.kv_cache_append_rotary(part["q"] if heads else None, part["k"], part["v"],
                                  c["positions"].to(DEV), cs.to(DEV), c["slots"].to(DEV), *caches,
                                  interleaved=pairs, out=out)
    torch.cuda.synchronize()
    assert r is out
    pos = c["positions"].tolist()
    known = np.array([0 <= p < 500 for p in pos])
    held = known & np.array([0 <= s < c["blocks"] * bs for s in c["slots"].tolist()])
    assert held.sum() > T // 2 or T < 3
    if heads:
        ref = kvq4.rotate(C.to64(c["q"]), pos, cs.numpy(), pairs)
        bound = turned_bound(C.to64(c["q"]), cs.numpy(), pos, pairs, dt)
        err = np.abs(C.to64(r) - ref)[known]
        assert (err <= bound[known]).all()
        assert (C.to64(r)[~known] == 7.0).all()
        if rot < dim:
            assert torch.equal(r.cpu()[known][..., rot:], c["q"][known][..., rot:])
    ref = kvq4.rotate(C.to64(c["k"]), pos, cs.numpy(), pairs)
    bound = turned_bound(C.to64(c["k"]), cs.numpy(), pos, pairs, dt)
    s = c["slots"][torch.from_numpy(held)]
    got = caches[0][(s // bs).to(DEV), :, (s % bs).to(DEV)]
    assert (np.abs(C.to64(got) - ref[held]) <= bound[held]).all()
    assert torch.equal(caches[1][(s // bs).to(DEV), :, (s % bs).to(DEV)].cpu(), c["v"][held])
    # nothing else changed
    for i in (0, 1):
        before[i][(s // bs).to(DEV), :, (s % bs).to(DEV)] = caches[i][(s // bs).to(DEV), :,
                                                                      (s % bs).to(DEV)]
        assert torch.equal(before[i], caches[i])


@pytest.mark.parametrize("dim,rot,pairs,dt", [(128, 128, False, "bf16"), (80, 48, True, "f16"),
                                              (40, 40, False, "bf16"), (9, 4, False, "f32")])
def test_queries_turned_in_place(sv, dim, rot, pairs, dt):
    c = rows_case(50, 4, 2, dim, 16, dt, True, 3)
    cs = table(500, rot).to(DEV)
    wide = c["k"]._base.to(DEV)
    q, k, v = (wide.as_strided(c[n].size(), c[n].stride(), c[n].storage_offset()) for n in "qkv")
    kc, vc = (torch.zeros((c["blocks"], 2, 16, dim), dtype=C.DT[dt], device=DEV) for _ in range(2))
    args = (k, v, c["positions"].to(DEV), cs, c["slots"].to(DEV), kc, vc)
    apart = sv.kv_cache_append_rotary(q, *args, interleaved=pairs, out=q.clone())
    r = sv.kv_cache_append_rotary(q, *args, interleaved=pairs, out=q)
    torch.cuda.synchronize()
    assert r is q and torch.equal(q, apart)
    rest = torch.ones(wide.shape[1], dtype=torch.bool)
    rest[8:8 + 4 * dim] = False                       # the other parts of the rows
    assert torch.equal(wide.cpu()[:, rest], c["k"]._base[:, rest])


def test_rows_off_16_bytes_take_the_element_path(sv):
    c = rows_case(60, 4, 2, 64, 16, "bf16", False, 5, extra=1)
    cs = table(500, 64)
    wide = c["k"]._base.to(DEV)
    q, k, v = (wide.as_strided(c[n].size(), c[n].stride(), c[n].storage_offset()) for n in "qkv")
    kc, vc = (torch.zeros((c["blocks"], 2, 16, 64), dtype=torch.bfloat16, device=DEV)
              for _ in range(2))
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    pos, slots = c["positions"].to(DEV), c["slots"].to(DEV)
    a = sv.kv_cache_append_rotary(q, k, v, pos, cs.to(DEV), slots, kc, vc, out=torch.zeros_like(q.contiguous()))
    odd = torch.zeros(cs.numel() + 1, device=DEV)[1:].view(cs.shape)     # a table off 16 bytes
    odd.copy_(cs)
    b = sv.kv_cache_append_rotary(q.contiguous(), k.contiguous(), v.contiguous(), pos, odd, slots,
                                  kc2, vc2, out=torch.zeros_like(a))
    c2 = sv.kv_cache_append_rotary(q.contiguous(), k.contiguous(), v.contiguous(), pos, cs.to(DEV),
                                   slots, kc2, vc2, out=torch.zeros_like(a))
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c2)
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_infinities_and_nan_pass(sv):
    """A row's own values, and no other row's."""
    c = rows_case(20, 2, 2, 64, 16, "bf16", False, 6)
    c["positions"][:] = torch.arange(20, dtype=torch.int32)
    c["slots"][:] = torch.arange(20)
    bad = c["k"]._base.clone()
    bad[4, ::5] = float("inf")
    bad[9, ::3] = float("nan")
    cs = table(500, 64).to(DEV)
    res = []
    for wide in (c["k"]._base.to(DEV), bad.to(DEV)):
        q, k, v = (wide.as_strided(c[n].size(), c[n].stride(), c[n].storage_offset()) for n in "qkv")
        kc, vc = (torch.zeros((c["blocks"], 2, 16, 64), dtype=torch.bfloat16, device=DEV)
                  for _ in range(2))
        res.append((sv.kv_cache_append_rotary(q, k, v, c["positions"].to(DEV), cs, c["slots"].to(DEV),
                                              kc, vc), kc, vc))
    torch.cuda.synchronize()
    rows = [i for i in range(20) if i not in (4, 9)]
    assert torch.equal(res[0][0][rows], res[1][0][rows])
    assert not torch.isfinite(res[1][0][4]).all() and not torch.isfinite(res[1][0][9]).all()
    for i in (1, 2):
        a, b = (res[j][i].transpose(1, 2).reshape(-1, 2, 64) for j in (0, 1))
        assert torch.equal(a[rows], b[rows])


def test_empty_calls_and_no_blocks(sv):
    cs = table(10, 64).to(DEV)
    e = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    i = torch.zeros(0, dtype=torch.int32, device=DEV)
    kc = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16, device=DEV)
    sv.kv_cache_append_rotary(e, e, e, i, cs, i.long(), kc, kc.clone())
    x = torch.randn((3, 2, 64), device=DEV).bfloat16()
    pos = torch.tensor([0, 5, 9], dtype=torch.int32, device=DEV)
    slots = torch.zeros(3, dtype=torch.int64, device=DEV)
    r = sv.kv_cache_append_rotary(x, x, x, pos, cs, slots, kc[:0], kc[:0])   # the queries alone
    full = sv.kv_cache_append_rotary(x, x, x, pos, cs, torch.arange(3, device=DEV), kc, kc.clone())
    none = sv.kv_cache_append_rotary(x, x, x, pos, cs[:0], slots, kc, kc, out=torch.ones_like(x))
    torch.cuda.synchronize()
    assert torch.equal(r, full) and (none == 1).all() and torch.equal(r[0], x[0])


def test_captured_and_on_another_stream(sv):
    c = rows_case(70, 8, 2, 128, 16, "bf16", True, 8)
    cs = table(500, 128).to(DEV)
    wide = c["k"]._base.to(DEV)
    q, k, v = (wide.as_strided(c[n].size(), c[n].stride(), c[n].storage_offset()) for n in "qkv")
    pos, slots = c["positions"].to(DEV), c["slots"].to(DEV)
    kc, vc = (torch.zeros((c["blocks"], 2, 16, 128), dtype=torch.bfloat16, device=DEV)
              for _ in range(2))
    out = torch.zeros((70, 8, 128), dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            sv.kv_cache_append_rotary(q, k, v, pos, cs, slots, kc, vc, out=out)
    for rep in range(4):
        wide.normal_()
        pos.copy_(torch.randint(0, 500, (70,), dtype=torch.int32))
        kc2, vc2 = kc.clone(), vc.clone()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(s):
            eager = sv.kv_cache_append_rotary(q, k, v, pos, cs, slots, kc2, vc2)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
