"""GPU parity of kv_blocktable_extend and kv_cache_append with the oracle, bit
for bit: ragged and empty requests, refused sequences, a short pool, freed
blocks taken back, batches of several scan passes, padded rows, in-place
lengths, graph capture."""

import numpy as np
import pytest
import torch

from oracle import pagedkv
from tests.kvcases import DEV, DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_token_verification_amd as m
    m.library()
    return m


def _state(B, bs, ctx, new, seed, pool=None, bad=0.0, freed=0, extra=2, ids_from=0):
    """Random tables, lengths and a pool; ``bad``: share of requests made invalid."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(ctx[0], ctx[1] + 1, B)
    n = rng.integers(new[0], new[1] + 1, B)
    width = -(-int((lens + n).max(initial=1)) // bs) + extra
    need = -(-lens // bs)
    ids = rng.permutation(ids_from + np.arange(int(need.sum()) + 10 ** 4 + B * freed))
    table = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    for b in range(B):
        if rng.random() < bad:
            n[b] = rng.choice([-1, -2 ** 31, width * bs - lens[b] + 1, 2 ** 31 - 1])
    want = int((-(-(lens + np.clip(n, 0, width * bs)) // bs) - need).sum())
    count = want + 5 if pool is None else pool
    free = np.full(max(count, 0) + B * freed + 7, -5, dtype=np.int32)
    free[:max(count, 0)] = ids[at:at + max(count, 0)] if count <= len(ids) - at else \
        ids_from + 10 ** 6 + np.arange(count)
    fr = nf = None
    if freed:
        fr = rng.integers(2 * 10 ** 6, 3 * 10 ** 6, (B, freed)).astype(np.int32)
        nf = rng.integers(-1, freed + 1, B).astype(np.int32)
    return dict(table=table, lens=lens.astype(np.int32), new=n.astype(np.int32), free=free,
                count=np.array([count], dtype=np.int32), freed=fr, num_freed=nf)


def _gpu(s):
    return {k: None if v is None else torch.from_numpy(v).to(DEV) for k, v in s.items()}


def _compare(sv, s, bs, T, in_place=False, out=None):
    g = _gpu(s)
    if in_place:
        B = len(s["lens"])
        e = lambda n, dt=torch.int32: torch.full((n,), 99, dtype=dt, device=DEV)  # noqa: E731
        out = dict(new_lens=g["lens"], num_taken=e(B), free_left=g["count"], cu_tokens=e(B + 1),
                   slot_map=e(T, torch.int64), positions=e(T))
    r = sv.kv_blocktable_extend(g["table"], g["lens"], g["new"], g["free"], g["count"], bs, T,
                                freed_blocks=g["freed"], num_freed=g["num_freed"], out=out)
    torch.cuda.synchronize()
    ref = pagedkv.blocktable_extend(s["table"], s["lens"], s["new"], s["free"], s["count"][0], bs,
                                    T, s["freed"], s["num_freed"])
    for key in ("new_lens", "num_taken", "cu_tokens", "slot_map", "positions"):
        assert np.array_equal(r[key].cpu().numpy(), ref[key]), key
    assert int(r["free_left"]) == ref["free_left"]
    assert np.array_equal(g["table"].cpu().numpy(), ref["block_table"])
    top = s["count"][0] if s["freed"] is None else len(s["free"])
    assert np.array_equal(g["free"].cpu().numpy()[:top], ref["free_blocks"][:top])
    return r, ref


CASES = [
    # (B, block size, contexts, new tokens, kwargs, rows beyond the tokens)
    (1, 16, (1000, 1000), (1, 1), {}, 0),
    (1, 1, (0, 0), (1, 1), {}, 0),                        # pages of one slot
    (3, 5, (0, 30), (0, 9), {}, 4),                       # odd pages, empty requests, padding
    (256, 16, (512, 4096), (9, 9), dict(freed=1), 0),     # a verification step
    (64, 16, (0, 0), (1, 700), {}, 33),                   # prompts: the fill launch of its own
    (64, 7, (3, 50), (0, 400), dict(bad=0.2, freed=2), 33),
    (1030, 16, (0, 60), (0, 5), dict(freed=1, bad=0.1), 9),   # two passes of the scans
    (2500, 3, (0, 20), (0, 9), dict(bad=0.05), 100),      # three, and the fill launch
    (40, 16, (0, 100), (0, 40), dict(pool=11), 0),        # a short pool
    (40, 16, (0, 100), (0, 40), dict(pool=0), 0),
    (40, 16, (0, 100), (0, 40), dict(pool=-3), 0),        # an invalid count is an empty pool
    (1200, 4, (0, 9), (0, 6), dict(pool=700, freed=1, bad=0.1), 5),
]


@pytest.mark.parametrize("in_place", [False, True], ids=["out", "inplace"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"B{c[0]}bs{c[1]}new{c[3][0]}-{c[3][1]}"
                         + "".join(sorted(c[4])))
def test_extend_parity(sv, case, in_place):
    B, bs, ctx, new, kw, pad = case
    for seed in range(3):
        s = _state(B, bs, ctx, new, seed, **kw)
        T = int(np.clip(s["new"].astype(np.int64), 0, 500).sum()) + pad
        _compare(sv, s, bs, T, in_place)


def test_extend_rows_short_of_the_tokens(sv):
    """Tokens beyond max_tokens refuse their sequence and every later one with any."""
    s = _state(20, 16, (0, 50), (1, 30), 5)
    for T in (0, 1, 100, 299):
        r, ref = _compare(sv, s, 16, T)
        assert (ref["num_taken"] == -1).any() and int(r["cu_tokens"][-1]) <= T


def test_extend_freed_beyond_the_stack(sv):
    s = _state(30, 16, (10, 50), (1, 1), 6, freed=3)
    s["free"] = s["free"][:int(s["count"][0]) + 4].copy()   # room for four of them
    _compare(sv, s, 16, 30)


def test_extend_empty_batch(sv):
    e = torch.zeros(0, dtype=torch.int32, device=DEV)
    r = sv.kv_blocktable_extend(torch.zeros((0, 4), dtype=torch.int32, device=DEV), e, e,
                                torch.arange(5, dtype=torch.int32, device=DEV),
                                torch.tensor([3], dtype=torch.int32, device=DEV), 16, 6)
    torch.cuda.synchronize()
    assert r["cu_tokens"].tolist() == [0] and r["free_left"].tolist() == [3]
    assert (r["slot_map"] == -1).all() and (r["positions"] == -1).all()


def test_extend_slots_pass_32_bits(sv):
    """Block ids near 2^31 with large pages: slots need 64 bits."""
    s = _state(4, 64, (100, 200), (30, 70), 7, ids_from=2 ** 31 - 3 * 10 ** 4)
    r, _ = _compare(sv, s, 64, int(s["new"].sum()))
    assert int(r["slot_map"].max()) > 2 ** 36


def test_extend_undoes_truncate_on_the_gpu(sv):
    """Truncate, then extend by the same amounts from an empty pool and the freed
    lists: the lengths come back and the tables hold the same blocks."""
    s = _gpu(_state(50, 16, (40, 300), (1, 1), 8))
    t0, l0 = s["table"].clone(), s["lens"].clone()
    drop = torch.randint(0, 40, (50,), generator=torch.Generator().manual_seed(1)).to(DEV, torch.int32)
    freed, nf = sv.kv_blocktable_truncate(s["table"], s["lens"], drop, 16, 4)
    r = sv.kv_blocktable_extend(s["table"], s["lens"], drop,
                                torch.full((200,), -9, dtype=torch.int32, device=DEV),
                                torch.zeros(1, dtype=torch.int32, device=DEV), 16,
                                int(drop.sum()), freed_blocks=freed, num_freed=nf)
    torch.cuda.synchronize()
    assert torch.equal(r["new_lens"], l0) and int(r["free_left"]) == 0
    assert torch.equal(s["table"].flatten().sort().values, t0.flatten().sort().values)
    assert torch.equal(s["table"] >= 0, t0 >= 0)


def test_extend_captured_step_advances_in_place(sv):
    """A captured in-place call replayed: each replay grows the same state further,
    as eager calls on a copy do."""
    s = _state(33, 16, (0, 90), (1, 9), 9, pool=300, extra=40)
    g, e = _gpu(s), _gpu(s)
    T = int(s["new"].sum()) + 6

    def outs(st):
        z = lambda n, dt=torch.int32: torch.zeros(n, dtype=dt, device=DEV)  # noqa: E731
        return dict(new_lens=st["lens"], num_taken=z(33), free_left=st["count"], cu_tokens=z(34),
                    slot_map=z(T, torch.int64), positions=z(T))

    def call(st, o):
        return sv.kv_blocktable_extend(st["table"], st["lens"], st["new"], st["free"], st["count"],
                                       16, T, out=o)
    og, oe = outs(g), outs(e)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            call(g, og)
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        call(e, oe)
        torch.cuda.synchronize()
        for k in oe:
            assert torch.equal(og[k], oe[k]), k
        assert torch.equal(g["table"], e["table"])


# ---------------------------------------------------------------------------
# append

APPEND = [
    # (T, kv_heads, dim, block size, dtype, fused rows)
    (1, 8, 128, 16, "bf16", True),
    (37, 1, 8, 1, "f32", False),
    (100, 5, 80, 24, "f16", True),
    (65, 3, 40, 7, "bf16", True),
    (300, 8, 256, 64, "f16", False),
    (129, 2, 129, 16, "bf16", False),    # no 16-byte rows
    (40, 3, 5, 3, "f32", True),
    (2304, 8, 128, 16, "bf16", True),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"T{c[0]}kv{c[1]}d{c[2]}bs{c[3]}{c[4]}")
def test_append_parity(sv, case):
    T, kv, dim, bs, dt, fused = case
    g = torch.Generator().manual_seed(T)
    nb = -(-2 * T // bs) + 2
    lead = 8 if fused else 0
    rows = torch.randn((T, lead + 2 * kv * dim), generator=g).to(DT[dt])
    both = torch.randn((nb, 2, kv, bs, dim), generator=g).to(DT[dt])
    slots = torch.randperm(nb * bs, generator=g)[:T]
    slots[::7] = torch.tensor([-1, -2 ** 62, nb * bs, 2 ** 40, 2 ** 32 + 3])[
        torch.arange(len(slots[::7])) % 5]
    gr, gb, gs = rows.to(DEV), both.to(DEV), slots.to(DEV)
    k, v = gr[:, lead:lead + kv * dim].view(T, kv, dim), gr[:, lead + kv * dim:].view(T, kv, dim)
    caches = (gb[:, 0], gb[:, 1]) if fused else (gb[:, 0].contiguous(), gb[:, 1].contiguous())
    sv.kv_cache_append(k, v, gs, *caches)
    torch.cuda.synchronize()
    bits = torch.int16 if DT[dt].itemsize == 2 else torch.int32
    for i, c in enumerate(caches):
        ref = pagedkv.cache_append(
            rows[:, lead + i * kv * dim:lead + (i + 1) * kv * dim].reshape(T, kv, dim)
            .view(bits).numpy(), slots.tolist(), both[:, i].contiguous().view(bits).numpy())
        assert np.array_equal(c.contiguous().cpu().view(bits).numpy(), ref), i


def test_append_unaligned_rows(sv):
    """Rows and caches off 16-byte boundaries take the element path."""
    base = torch.randn(2 * 9 * 64 + 1, device=DEV).to(torch.bfloat16)
    k = base[1:1 + 9 * 64].view(9, 1, 64)
    v = base[9 * 64:18 * 64].view(9, 1, 64)
    c = torch.zeros(2 * 4 * 16 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:]
    kc, vc = c[:4096].view(4, 1, 16, 64), c[4096:].view(4, 1, 16, 64)
    slots = torch.arange(5, 14, device=DEV)
    sv.kv_cache_append(k, v, slots, kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc.view(64, 64)[5:14], k[:, 0]) and torch.equal(vc.view(64, 64)[5:14], v[:, 0])
    assert (kc.view(64, 64)[:5] == 0).all() and (kc.view(64, 64)[14:] == 0).all()


def test_append_empty(sv):
    c = torch.zeros((2, 1, 16, 64), device=DEV)
    z = torch.zeros((0, 1, 64), device=DEV)
    sv.kv_cache_append(z, z, torch.zeros(0, dtype=torch.int64, device=DEV), c, c.clone())
    torch.cuda.synchronize()
    assert (c == 0).all()


def test_append_cache_beyond_32_bit_offsets(sv):
    """A cache of more than 2^32 bytes: the last slots are reached."""
    nb, kv, bs, dim = 2 ** 15 + 3, 8, 64, 160
    k_cache = torch.zeros((nb, kv, bs, dim), dtype=torch.bfloat16, device=DEV)
    assert k_cache.numel() * 2 > 2 ** 32
    v_cache = torch.zeros((nb, kv, bs, dim), dtype=torch.bfloat16, device=DEV)
    k = torch.randn((3, kv, dim), device=DEV).to(torch.bfloat16)
    slots = torch.tensor([nb * bs - 1, 0, (nb - 2) * bs + 5], device=DEV)
    sv.kv_cache_append(k, -k, slots, k_cache, v_cache)
    torch.cuda.synchronize()
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(k_cache[s // bs, :, s % bs], k[t])
        assert torch.equal(v_cache[s // bs, :, s % bs], -k[t])
    assert int((k_cache != 0).sum()) == int((k != 0).sum())


