"""GPU parity of kv_paged_attention_q4 at calls that its other tests leave out, within
bounds by arithmetic (tests/kvq4cases.py)."""

import math

import numpy as np
import pytest
import torch

from tests import kvcases as C
from tests import kvq4cases as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_token_verification_amd as m
    m.library()
    return m


def _args(g):
    return [g[n] for n in Q.NAMES]


def _run(sv, case, **kw):
    r = sv.kv_paged_attention_q4(*_args(Q.on_gpu(case)), lse=True, **kw)
    torch.cuda.synchronize()
    return r


def _parity(sv, case, dtype, note="", **kw):
    r = _run(sv, case, **kw)
    ref = Q.reference(case, kw.get("scale"), kw.get("sliding_window", 0))
    return Q.check(C.to64(r["out"]), C.to64(r["lse"]), ref, dtype, case["q"].shape[2], note)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 256])
def test_every_configuration(sv, dim, dtype):
    """Each tile of each head size, whole and padded: short and split keys, windows."""
    case = Q.attend_case([20, 0, 1500, 260], [2, 30, 5, 11], 8, 1, dim, 16, dtype, seed=dim)
    for window in (0, 300):
        ref = Q.reference(case, None, window)
        for hint in (2, 4, 6, 30):          # 16, 32, 48 and 64 rows
            r = _run(sv, case, max_new=hint, sliding_window=window)
            Q.check(C.to64(r["out"]), C.to64(r["lse"]), ref, dtype, dim, (hint, window))


@pytest.mark.parametrize("ctx,new,heads,dim,dtype,hint", [
    (60, 140, 256, 64, "bf16", 1),       # 9 tiles of 16 rows for 4 places a head
    (10, 200, 128, 128, "f16", 0),
    (9, 150, 256, 256, "bf16", 0)])      # 3 tiles of 64 rows for 2
def test_one_sequence_of_more_tiles_than_places(sv, ctx, new, heads, dim, dtype, hint):
    """A single sequence whose tiles alone fill the chip, on a table so wide that its
    keys could be split."""
    case = Q.attend_case([ctx], [new], heads, heads, dim, 16, dtype, seed=31)
    wide = torch.full((1, 600), -1, dtype=torch.int32)
    wide[:, :case["block_table"].shape[1]] = case["block_table"]
    _parity(sv, {**case, "block_table": wide}, dtype, max_new=hint)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("gap", [8.0, 12.0, 16.0])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_flat_tail_behind_a_dominant_key(sv, dtype, gap, dim):
    """Every key but the first scores ``gap`` below it and has value 1: the output is
    the tail's share, p w / (1 + p w) at position p, w = exp(-gap)."""
    T, bs, heads, kv = 1500, 16, 2, 1
    case = Q.attend_case([0], [T], heads, kv, dim, bs, dtype, seed=dim, poison=False)
    k, v = np.zeros((T, dim), np.float32), np.ones((T, dim), np.float32)
    k[0, 1], v[0] = gap, 0.0
    rows = Q.quantised(torch.from_numpy(k), torch.from_numpy(v))
    page, at = case["block_table"][0, torch.arange(T) // bs].long(), torch.arange(T) % bs
    for n, t in rows.items():
        for h in range(kv):
            case["cache"][n][page, h, at] = t
    case["q"] = torch.zeros_like(case["q"])
    case["q"][:, :, 1] = 1.0
    ref = Q.reference(case, 1.0)
    p = np.arange(T)[:, None, None] * math.exp(-gap)
    unit = float(rows["v_scales"][1]) * 6          # 1 as the cache holds it
    assert np.abs(ref["out"] / np.maximum(unit * p / (1 + p), 1e-30) - 1)[1:].max() < 1e-9
    r = _run(sv, case, scale=1.0, max_new=T)
    share = Q.check(C.to64(r["out"]), C.to64(r["lse"]), ref, dtype, dim)
    print(f"{share:.3f} of the bound")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ctx,new", [([100], [1]), ([6000, 40], [2, 40])])
def test_values_near_the_largest(sv, dim, ctx, new):
    """Units of 4e37 (values to 2.4e38): a late key that outweighs the ones before it
    leaves the sums finite."""
    case = Q.attend_case(ctx, new, 2, 1, dim, 16, "bf16", seed=33)
    case["q"] = torch.zeros_like(case["q"])
    case["q"][:, :, 0] = 1.0
    c = case["cache"]
    for b, L in enumerate(case["seq_lens"].tolist()):
        pos = torch.arange(L)
        page, at = case["block_table"][b, pos // 16].long(), pos % 16
        c["k_codes"][page, 0, at, 0] &= 0xf0              # channel 0: zero
        last = case["block_table"][b, (ctx[b] - 1) // 16].long(), 0, (ctx[b] - 1) % 16
        c["k_codes"][last][0] |= 7                        # 6
        c["k_scales"][last][0] = 127
        c["v_scales"][page, 0, at] = 4e37
    _parity(sv, case, "bf16", scale=1.0)


def test_units_of_keys_far_from_one(sv):
    for k_std, q_std, scale in ((1e25, 1e-25, None), (1e-30, 1e25, 1e4), (3e-38, 1.0, 1e30)):
        case = Q.attend_case([300, 7], [4, 20], 4, 2, 128, 16, "bf16", seed=5, q_std=q_std, k_std=k_std)
        _parity(sv, case, "bf16", (k_std, q_std), scale=scale)


@pytest.mark.parametrize("dim", [32, 96, 160, 192, 224])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_long_contexts_of_head_sizes_between(sv, dim, dtype):
    for i, (ctx, new, heads, kv, bs) in enumerate([
            ([3000, 5], [1, 1], 4, 2, 16), ([70, 400], [9, 20], 2, 2, 24), ([10, 700], [150, 60], 4, 2, 32),
            ([2500], [130], 2, 1, 16)]):
        case = Q.attend_case(ctx, new, heads, kv, dim, bs, dtype, seed=60 + i)
        _parity(sv, case, dtype, (i, dim), max_new=max(new))


def test_reused_outputs_take_any_hint_and_window(sv):
    """One out dict over calls whose hint and window ask for larger workspaces, in any
    order; a call captured with the first workspace still replays right."""
    case = Q.attend_case([9000, 5000, 40, 7], [10, 10, 10, 10], 32, 8, 128, 16, "bf16", seed=34)
    args = _args(Q.on_gpu(case))
    out = sv.kv_paged_attention_q4(*args, max_new=1)
    first = out["workspace"]
    alone = out["out"].clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            sv.kv_paged_attention_q4(*args, max_new=1, out=out)
    del first
    grown = set()
    for hint, window in ((1, 0), (9, 0), (40, 0), (1, 512), (9, 512), (40, 300), (0, 0), (9, 0)):
        fresh = sv.kv_paged_attention_q4(*args, max_new=hint, sliding_window=window)
        r = sv.kv_paged_attention_q4(*args, max_new=hint, sliding_window=window, out=out)
        torch.cuda.synchronize()
        assert r is out and torch.equal(r["out"], fresh["out"]), (hint, window)
        grown.add(r["workspace"].numel())
        junk = [torch.full((n,), 0x7f, dtype=torch.uint8, device=C.DEV) for n in sorted(grown)]
        out["out"].fill_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["out"], alone), (hint, window)
        assert all((j == 0x7f).all() for j in junk)
        del junk
    # an explicit workspace is the caller's, sized by its own call
    need = sv.kv_paged_attention_q4_workspace_bytes(args[0], args[1], args[2], max_new=1)
    assert need > 0
    enough = torch.empty(need, dtype=torch.uint8, device=C.DEV)
    sv.kv_paged_attention_q4(*args, max_new=1, out=out, workspace=enough)
    torch.cuda.synchronize()
    assert torch.equal(out["out"], alone)
    with pytest.raises(sv.SpecVerifyError, match="workspace has"):
        sv.kv_paged_attention_q4(*args, max_new=1, out=out, workspace=enough[:need - 256])


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f16", 128), ("bf16", 256)])
def test_batches_of_thousands(sv, dtype, dim):
    """Single tokens and short windows of 5000 sequences, one long one among them: more
    than a workgroup's threads hold."""
    rng = np.random.default_rng(35)
    ctx, new = rng.integers(0, 30, 5000).tolist(), rng.integers(0, 3, 5000).tolist()
    ctx[4321], new[4321] = 3000, 2
    case = Q.attend_case(ctx, new, 2, 1, dim, 16, dtype, seed=35)
    _parity(sv, case, dtype, max_new=2)


def test_rows_of_no_sequence_stay(sv):
    case = Q.attend_case([100, 4000], [3, 2], 8, 2, 128, 16, "bf16", seed=36, lead=5, tail=7)
    g = Q.on_gpu(case)
    out = dict(out=torch.full((17, 8, 128), 7.0, dtype=torch.bfloat16, device=C.DEV),
               lse=torch.full((17, 8), 7.0, device=C.DEV), workspace=None)
    sv.kv_paged_attention_q4(*_args(g), out=out)
    torch.cuda.synchronize()
    for rows in (slice(0, 5), slice(10, 17)):
        assert (out["out"][rows] == 7.0).all() and (out["lse"][rows] == 7.0).all()
    Q.check(C.to64(out["out"]), C.to64(out["lse"]), Q.reference(case), "bf16", 128)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_that_see_nothing_and_missing_pages(sv, dtype, dim):
    """Lengths below the tokens', pages without a block or with one past the cache, in
    the first, the middle and the last units, of short and of split keys."""
    case = Q.attend_case([30, 700, 3, 5000, 200], [9, 20, 6, 3, 130], 4, 2, dim, 16, dtype, seed=38)
    table, lens = case["block_table"], case["seq_lens"]
    nb = case["cache"]["k_codes"].shape[0]
    lens[0], lens[2] = 4, 0                       # 35 rows before position 0, a whole sequence
    table[1, 0], table[1, 5], table[1, 20:24], table[1, -1] = -1, nb, -5, 2 ** 31 - 1
    table[3, 100:130] = -1
    table[3, 300], table[3, 313:] = nb + 7, -1
    table[4] = -1                                 # nothing but missing pages
    for window in (0, 40):
        r = _run(sv, case, sliding_window=window)
        ref = Q.reference(case, None, window)
        Q.check(C.to64(r["out"]), C.to64(r["lse"]), ref, dtype, dim, window)
        none = torch.from_numpy(np.isneginf(ref["lse"]))
        assert none.sum() > 130 * 4
        assert (r["out"].cpu()[none] == 0).all() and torch.isneginf(r["lse"].cpu()[none]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256, 96])
def test_what_is_not_a_number_stays_where_it_is_seen(sv, dtype, dim):
    """A key, a value or a query that is not a number reaches the rows that see it, and
    leaves every other row as it was, bit for bit."""
    ctx, new, heads, kv = [40, 6000, 300], [9, 2, 30], 8, 2
    case = Q.attend_case(ctx, new, heads, kv, dim, 16, dtype, seed=39)
    clean = _run(sv, case)
    window = 50
    clean_w = _run(sv, case, sliding_window=window)
    cu = case["cu_tokens"].tolist()
    for b, pos in ((0, 45), (0, 3), (1, 0), (1, 3000), (1, 6001), (2, 310)):
        page, at = int(case["block_table"][b, pos // 16]), pos % 16
        for name, bad in (("k_scales", 255), ("v_scales", math.nan), ("v_scales", math.inf)):
            t = case["cache"][name]
            kept = t[page, 1, at].clone()
            t[page, 1, at] = bad
            for w, base in ((0, clean), (window, clean_w)):
                r = _run(sv, case, sliding_window=w)
                hit = torch.zeros((sum(new), heads), dtype=torch.bool)
                for j in range(new[b]):
                    p = ctx[b] + j
                    hit[cu[b] + j, 4:] = pos <= p and (w == 0 or pos > p - w)
                note = (b, pos, name, bad, w)
                out, lse = r["out"].cpu(), r["lse"].cpu()
                assert torch.isnan(out[hit]).all(), note
                assert torch.equal(out[~hit], base["out"].cpu()[~hit]), note
                assert torch.equal(lse[~hit], base["lse"].cpu()[~hit]), note
                if name == "k_scales":
                    assert torch.isnan(lse[hit]).all(), note
            t[page, 1, at] = kept
    for bad in (math.nan, math.inf, -math.inf):
        dirty = {**case, "q": case["q"].clone()}
        hit = torch.zeros((sum(new), heads), dtype=torch.bool)
        for t, h in ((2, 1), (9, 7), (10, 0), (25, 4)):
            dirty["q"][t, h, dim // 2 + 3] = bad
            hit[t, h] = True
        r = _run(sv, dirty)
        assert torch.isnan(r["out"].cpu()[hit]).all() and torch.isnan(r["lse"].cpu()[hit]).all()
        assert torch.equal(r["out"].cpu()[~hit], clean["out"].cpu()[~hit])
        assert torch.equal(r["lse"].cpu()[~hit], clean["lse"].cpu()[~hit])


def test_empty_calls_and_no_pages(sv):
    case = Q.on_gpu(Q.attend_case([30], [4], 4, 2, 64, 16, "bf16"))
    i32 = dict(dtype=torch.int32, device=C.DEV)
    r = sv.kv_paged_attention_q4(case["q"][:0], case["cache"], case["block_table"], case["seq_lens"],
                                 torch.zeros(2, **i32))
    assert r["out"].shape == (0, 4, 64)
    r = sv.kv_paged_attention_q4(case["q"], case["cache"], torch.zeros((0, 3), **i32),
                                 torch.zeros(0, **i32), torch.zeros(1, **i32))
    assert r["out"].shape == (4, 4, 64)
    for table in (torch.zeros((1, 0), **i32), torch.full((1, 4), -1, **i32)):
        r = sv.kv_paged_attention_q4(case["q"], case["cache"], table, case["seq_lens"],
                                     case["cu_tokens"], lse=True)
        torch.cuda.synchronize()
        assert (r["out"] == 0).all() and torch.isneginf(r["lse"]).all()
    none = sv.make_kv_cache_q4(0, 2, 16, 64, device=C.DEV)
    r = sv.kv_paged_attention_q4(case["q"], none, case["block_table"], case["seq_lens"],
                                 case["cu_tokens"], lse=True)
    torch.cuda.synchronize()
    assert (r["out"] == 0).all() and torch.isneginf(r["lse"]).all()


def test_overlapping_token_ranges_compute_nothing(sv):
    """Offsets that do not ascend ask for more tiles than the launch was sized for."""
    case = Q.on_gpu(Q.attend_case([540] * 12, [1] * 12, 4, 2, 128, 16, "bf16"))
    q = torch.randn((160, 4, 128), device=C.DEV).bfloat16()
    cu = torch.tensor([160 * (i % 2) for i in range(13)], dtype=torch.int32, device=C.DEV)
    out = dict(out=torch.full_like(q, 3.0), lse=None, workspace=None)
    sv.kv_paged_attention_q4(q, case["cache"], case["block_table"], case["seq_lens"] + 159, cu,
                             out=out, max_new=160)
    torch.cuda.synchronize()
    assert (out["out"] == 3.0).all()


def test_rows_beyond_32_bits(sv):
    """Row numbers above 2^31 and byte offsets far above 2^32: the last pages of a cache
    of 70 GB, by whole pages and by the position."""
    bs, kv, dim, nb = 32, 2, 32, (1 << 25) + (1 << 20)
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("not enough memory")
    case = Q.attend_case([400, 3], [3, 40], 4, kv, dim, bs, "bf16", seed=41, poison=False)
    small, used = case["cache"], case["block_table"] >= 0
    n = small["k_codes"].shape[0]
    g = Q.on_gpu(case)
    big = {name: torch.empty((nb, *t.shape[1:]), dtype=t.dtype, device=C.DEV) for name, t in small.items()}
    for name, t in small.items():
        big[name][nb - n:] = t.to(C.DEV)
    table = torch.where(used, case["block_table"] + (nb - n), -1)
    plain = sv.kv_paged_attention_q4(*_args(g), lse=True)
    far = sv.kv_paged_attention_q4(g["q"], big, table.to(C.DEV), g["seq_lens"], g["cu_tokens"], lse=True)
    torch.cuda.synchronize()
    assert torch.equal(plain["out"], far["out"]) and torch.equal(plain["lse"], far["lse"])
    Q.check(C.to64(far["out"]), C.to64(far["lse"]), Q.reference(case), "bf16", dim)
    del big
    torch.cuda.empty_cache()


def test_graphs_that_share_a_workspace_and_another_stream(sv):
    """Two captured calls with one workspace, replayed in turn with new inputs, and
    eager calls of other streams between them."""
    cases = [Q.attend_case([6000, 30, 2000], [5, 9, 1], 8, 2, 128, 16, "bf16", seed=s) for s in (1, 2)]
    on = [Q.on_gpu(c) for c in cases]
    outs = [sv.kv_paged_attention_q4(*_args(g), lse=True) for g in on]
    outs[1]["workspace"] = outs[0]["workspace"]
    graphs = []
    for g, o in zip(on, outs):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(graph, stream=s):
                sv.kv_paged_attention_q4(*_args(g), out=o)
        graphs.append(graph)
    gen = torch.Generator().manual_seed(3)
    streams = [torch.cuda.Stream() for _ in on]
    for rep in range(5):
        for i, g in enumerate(on):
            g["q"].copy_(torch.randn(g["q"].shape, generator=gen).to(torch.bfloat16))
            outs[i]["out"].fill_(9.0)
        torch.cuda.synchronize()
        graphs[rep % 2].replay()
        graphs[1 - rep % 2].replay()
        torch.cuda.synchronize()
        eager = []
        for st, g in zip(streams, on):           # at once, each with its own workspace
            with torch.cuda.stream(st):
                eager.append(sv.kv_paged_attention_q4(*_args(g), lse=True))
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert torch.equal(o["out"], e["out"]) and torch.equal(o["lse"], e["lse"]), rep
    for c, g, o in zip(cases, on, outs):
        ref = Q.reference({**c, "q": g["q"].cpu()})
        Q.check(C.to64(o["out"]), C.to64(o["lse"]), ref, "bf16", 128)


def test_one_block_held_by_two_sequences(sv):
    """Sequences that share a prefix's blocks, and a table that names a block twice."""
    case = Q.attend_case([200, 200], [4, 9], 4, 2, 64, 16, "f16", seed=42)
    case["block_table"][1, :12] = case["block_table"][0, :12]
    case["block_table"][0, 3] = case["block_table"][0, 2]
    _parity(sv, case, "f16")
