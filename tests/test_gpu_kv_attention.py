"""GPU parity of kv_paged_attention with the float64 oracle, within bounds by
arithmetic (tests/kvcases.py).  Every slot that no sequence holds is NaN or
infinite, so a value read from a masked place shows."""

import numpy as np
import pytest
import torch

from tests import kvcases as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_token_verification_amd as m
    m.library()
    return m


def _run(sv, case, **kw):
    g = C.on_gpu(case)
    r = sv.kv_paged_attention(g["q"], g["k_cache"], g["v_cache"], g["block_table"], g["seq_lens"],
                              g["cu_tokens"], lse=True, **kw)
    torch.cuda.synchronize()
    return r


def _parity(sv, case, dtype, scale=None, window=0, **kw):
    r = _run(sv, case, scale=scale, sliding_window=window, **kw)
    ref = C.reference(case, scale, window)
    return C.check(C.to64(r["out"]), C.to64(r["lse"]), ref, dtype, case["q"].shape[2])


SHAPES = [
    # (contexts, new tokens, heads, kv_heads, head_dim, block size, window)
    ([0], [1], 1, 1, 64, 16, 0),                         # the smallest call
    ([1000], [1], 8, 2, 128, 16, 0),
    ([17, 0, 63, 200, 5], [1, 1, 1, 1, 1], 4, 4, 64, 16, 0),
    ([30, 0, 100], [5, 9, 1], 8, 2, 128, 16, 0),         # a drafted window
    ([64, 15, 33], [9, 9, 9], 12, 4, 128, 5, 0),         # groups of 3, odd pages
    ([40, 7], [9, 3], 14, 2, 64, 1, 0),                  # groups of 7, pages of one slot
    ([0, 3], [70, 45], 4, 2, 128, 24, 0),                # prompts, pages across tiles
    ([0], [200], 2, 2, 64, 32, 0),
    ([129], [130], 8, 1, 256, 16, 0),
    ([50, 0], [33, 65], 2, 1, 256, 64, 0),
    ([300, 10], [4, 40], 4, 2, 128, 16, 7),              # sliding windows
    ([300, 100, 0], [1, 1, 1], 4, 4, 64, 16, 64),
    ([500], [3], 16, 2, 256, 16, 1),                     # a token sees itself alone
    ([0, 20, 0, 9], [0, 3, 0, 0], 4, 2, 64, 16, 0),      # sequences without new tokens
    ([100], [6], 3, 3, 80, 16, 0),                       # other head sizes
    ([70, 9], [2, 20], 4, 2, 96, 16, 0),
    ([33], [5], 2, 1, 8, 16, 0),
    ([120], [7], 4, 1, 192, 16, 30),
    ([60, 2], [12, 5], 6, 2, 248, 9, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"c{s[0][0]}n{s[1][0]}h{s[2]}-{s[3]}"
                         f"d{s[4]}bs{s[5]}w{s[6]}")
def test_attention_parity(sv, shape, dtype):
    ctx, new, heads, kv, dim, bs, window = shape
    for seed, poison in ((1, float("nan")), (2, float("inf"))):
        case = C.attend_case(ctx, new, heads, kv, dim, bs, dtype, seed=seed, poison=poison,
                             fused=seed == 2)
        share = _parity(sv, case, dtype, window=window)
        print(f"{dtype} {shape}: {share:.3f} of the bound")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256, 72])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_split_keys_parity(sv, dtype, dim, new):
    """Few rows and long contexts: the key axis is split over workgroups and joined,
    beside a short sequence that is not."""
    if new == 40 and dim > 64:
        ctx = [2500, 10]
    else:
        ctx = [9001, 10, 4000]
    case = C.attend_case(ctx, [new] * len(ctx), 2, 1, dim, 16, dtype, seed=new)
    _parity(sv, case, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_peaked_and_large_scores(sv, dtype):
    """Scores of several hundred: the running maximum moves by much, most weights
    vanish."""
    for seed, std in ((1, 30.0), (2, 100.0)):
        case = C.attend_case([700, 20], [9, 40], 4, 2, 128, 16, dtype, seed=seed, q_std=std)
        _parity(sv, case, dtype)
    case = C.attend_case([700, 20], [9, 40], 4, 2, 128, 16, dtype, seed=3)
    _parity(sv, case, dtype, scale=1e-6)
    _parity(sv, case, dtype, scale=2.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_growing_scores(sv, dtype):
    """Keys whose scores grow along the sequence move the maximum at every tile."""
    case = C.attend_case([900], [5], 2, 1, 64, 16, dtype, seed=4)
    pos = torch.arange(905)
    ids = case["block_table"][0].long()
    direction = case["q"][2, 0].float()
    k = (pos[:, None] / 40.0) * direction / direction.norm()
    case["k_cache"][ids[pos // 16], 0, pos % 16] = k.to(case["k_cache"].dtype)
    _parity(sv, case, dtype)


@pytest.mark.parametrize("hint", [1, 5, 17, 60, 10 ** 6])
def test_every_tile_shape_is_right_for_every_batch(sv, hint):
    """max_new only picks the tile shape."""
    case = C.attend_case([40, 0, 333, 7], [1, 50, 9, 130], 8, 2, 128, 16, "bf16", seed=5)
    _parity(sv, case, "bf16", max_new=hint)
    _parity(sv, case, "bf16", max_new=hint, window=23)
    case = C.attend_case([40, 0, 333, 7], [1, 50, 9, 130], 6, 2, 64, 16, "f16", seed=6)
    _parity(sv, case, "f16", max_new=hint)
    case = C.attend_case([40, 7], [20, 70], 3, 3, 256, 16, "bf16", seed=7)
    _parity(sv, case, "bf16", max_new=hint)


def test_rows_of_no_sequence_are_left(sv):
    case = C.attend_case([30, 100], [4, 9], 4, 2, 128, 16, "bf16", seed=8, lead=3, tail=70)
    g = C.on_gpu(case)
    out = dict(out=torch.full_like(g["q"].contiguous(), 7.0),
               lse=torch.full((86, 4), 5.0, device=C.DEV), workspace=None)
    r = sv.kv_paged_attention(g["q"], g["k_cache"], g["v_cache"], g["block_table"], g["seq_lens"],
                              g["cu_tokens"], out=out)
    torch.cuda.synchronize()
    C.check(C.to64(r["out"]), C.to64(r["lse"]), C.reference(case), "bf16", 128)
    for rows in (slice(0, 3), slice(16, 86)):
        assert (r["out"][rows] == 7.0).all() and (r["lse"][rows] == 5.0).all()


@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "f16"), (256, "bf16"), (96, "f32")])
def test_rows_that_see_nothing(sv, dim, dtype):
    """Lengths shorter than the new tokens, zero lengths, pages off the cache and
    positions beyond the table."""
    case = C.attend_case([20, 0, 40, 300, 33], [5, 8, 4, 3, 40], 4, 2, dim, 16, dtype, seed=9)
    case["seq_lens"] = torch.tensor([25, 3, 0, 303, 73], dtype=torch.int32)
    case["block_table"][3, :2] = torch.tensor([-1, 10 ** 6])      # missing pages
    case["block_table"][4, 1] = -7
    _parity(sv, case, dtype)
    case["block_table"][3, :] = -1                                # no page at all
    _parity(sv, case, dtype)
    case["block_table"] = case["block_table"][:, :2].contiguous()  # positions beyond the table
    _parity(sv, case, dtype)
    _parity(sv, case, dtype, window=11)
    case["seq_lens"] = torch.tensor([-4, 0, -2 ** 31, 2 ** 31 - 1, 0], dtype=torch.int32)
    _parity(sv, case, dtype)


@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "f16"), (256, "bf16"), (128, "f32"),
                                       (80, "bf16")])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), float("-inf")])
def test_unseen_infinities_and_nan_stay_out(sv, dim, dtype, poison):
    """A later token's keys and values may hold anything: earlier rows of the same
    chunk, and rows whose window has passed it, come out as without it."""
    ctx, new, at = [70, 0], [40, 90], (85, 50)      # the poisoned position of each sequence
    case = C.attend_case(ctx, new, 4, 2, dim, 16, dtype, seed=10)
    clean = {k: v.clone() for k, v in case.items()}
    for b, p in enumerate(at):
        page = int(case["block_table"][b, p // 16])
        case["v_cache"][page, :, p % 16, ::3] = poison
        case["k_cache"][page, 0, p % 16, 5] = poison
    for window in (0, 10):
        ref = C.reference(clean, None, window)
        r = _run(sv, case, sliding_window=window)
        out, lse = C.to64(r["out"]), C.to64(r["lse"])
        for b, p in enumerate(at):
            t0 = int(case["cu_tokens"][b])
            for j in range(new[b]):
                pos = ctx[b] + j
                if pos >= p and not (window and pos >= p + window):
                    ref["lse"][t0 + j] = np.nan          # these rows see it
                    assert not np.isfinite(out[t0 + j, 2:, ::3]).any(), (b, j)
                    if poison == poison:                 # value columns it does not touch
                        assert np.isfinite(out[t0 + j, 2:, 1::3]).all(), (b, j)
        C.check(out, lse, ref, dtype, dim, (window, poison))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_query_row_stays_alone(sv, dtype):
    case = C.attend_case([70], [12], 4, 2, 128, 16, dtype, seed=11)
    case["q"][5, 1, 7] = float("nan")
    r = _run(sv, case)
    out = C.to64(r["out"])
    assert np.isnan(out[5, 1]).all()
    clean = {**case, "q": case["q"].clone()}
    clean["q"][5, 1, 7] = 0.0
    ref = C.reference(clean)
    ref["lse"][5, 1] = np.nan
    C.check(out, None, ref, dtype, 128)


def test_offsets_beyond_32_bits(sv):
    """A cache of more than 2^32 bytes whose sequence lives in its last pages."""
    nb, kv, bs, dim = 2 ** 16 + 40, 4, 64, 128
    case = C.attend_case([500], [9], 8, kv, dim, bs, "bf16", seed=12, spare=0)
    used = case["k_cache"].shape[0]
    big = {}
    for n in ("k_cache", "v_cache"):
        big[n] = torch.full((nb, kv, bs, dim), float("nan"), dtype=torch.bfloat16, device=C.DEV)
        assert big[n].numel() * 2 > 2 ** 32
        big[n][nb - used:] = case[n].to(C.DEV)
    table = torch.where(case["block_table"] >= 0, case["block_table"] + nb - used, -1)
    r = sv.kv_paged_attention(case["q"].to(C.DEV), big["k_cache"], big["v_cache"],
                              table.to(C.DEV), case["seq_lens"].to(C.DEV),
                              case["cu_tokens"].to(C.DEV), lse=True)
    torch.cuda.synchronize()
    C.check(C.to64(r["out"]), C.to64(r["lse"]), C.reference(case), "bf16", dim)


def test_many_sequences_and_many_tiles(sv):
    """More sequences than a pass of the work search, short ones beside long ones."""
    rng = np.random.default_rng(13)
    ctx = rng.integers(0, 40, 700).tolist()
    new = rng.integers(0, 4, 700).tolist()
    ctx[350], new[350] = 3000, 2
    case = C.attend_case(ctx, new, 2, 1, 64, 16, "bf16", seed=13)
    _parity(sv, case, "bf16")


def test_repeats_bit_for_bit_and_on_another_stream(sv):
    case = C.attend_case([5000, 80], [5, 30], 8, 2, 128, 16, "bf16", seed=14)
    g = C.on_gpu(case)
    args = (g["q"], g["k_cache"], g["v_cache"], g["block_table"], g["seq_lens"], g["cu_tokens"])
    a = sv.kv_paged_attention(*args, lse=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = sv.kv_paged_attention(*args, lse=True)
    s.synchronize()
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    # a workspace full of what another call left, and reused outputs
    a["workspace"].fill_(0xff)
    c = sv.kv_paged_attention(*args, out=a)
    torch.cuda.synchronize()
    assert c is a and torch.equal(a["out"], b["out"])


def test_empty_calls(sv):
    case = C.on_gpu(C.attend_case([20], [3], 4, 2, 64, 16, "bf16"))
    z = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=C.DEV)
    r = sv.kv_paged_attention(z, case["k_cache"], case["v_cache"], case["block_table"],
                              case["seq_lens"], torch.zeros(2, dtype=torch.int32, device=C.DEV))
    e = torch.zeros(0, dtype=torch.int32, device=C.DEV)
    sv.kv_paged_attention(case["q"], case["k_cache"], case["v_cache"], case["block_table"][:0], e,
                          case["cu_tokens"][:1])
    # no pages at all: every row is empty
    r = sv.kv_paged_attention(case["q"], case["k_cache"][:0], case["v_cache"][:0],
                              case["block_table"], case["seq_lens"], case["cu_tokens"], lse=True)
    torch.cuda.synchronize()
    assert (r["out"] == 0).all() and torch.isneginf(r["lse"]).all()
    # tables without columns
    r = sv.kv_paged_attention(case["q"], case["k_cache"], case["v_cache"],
                              case["block_table"][:, :0].contiguous(), case["seq_lens"],
                              case["cu_tokens"], lse=True)
    torch.cuda.synchronize()
    assert (r["out"] == 0).all() and torch.isneginf(r["lse"]).all()


def test_captured_graph_follows_the_lengths(sv):
    """One captured call replayed while lengths, tables and row counts move, with
    eager work between, against the eager call every time."""
    case = C.attend_case([4000, 60, 0], [4, 4, 4], 8, 2, 128, 16, "bf16", seed=15, tail=20,
                         poison=0.5)
    g = C.on_gpu(case)
    args = (g["q"], g["k_cache"], g["v_cache"], g["block_table"], g["seq_lens"], g["cu_tokens"])
    first = sv.kv_paged_attention(*args, lse=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            sv.kv_paged_attention(*args, out=first)
    for lens, cu in (([4004, 64, 4], [0, 4, 8, 12]), ([100, 64, 2], [0, 1, 9, 11]),
                     ([3500, 5, 0], [2, 22, 22, 32]), ([4004, 64, 4], [0, 4, 8, 12])):
        g["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        g["cu_tokens"].copy_(torch.tensor(cu, dtype=torch.int32))
        first["out"].fill_(3.0)
        first["lse"].fill_(3.0)
        eager = sv.kv_paged_attention(*args, out=dict(out=torch.full_like(first["out"], 3.0),
                                                      lse=torch.full_like(first["lse"], 3.0),
                                                      workspace=None))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first["out"], eager["out"]) and torch.equal(first["lse"], eager["lse"])


@pytest.mark.parametrize("short", [False, True])
@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("bf16", 128), ("f16", 256), ("f32", 64)])
def test_windows_of_any_width(sv, dtype, dim, short):
    """The widest windows; short: also rows before position 0 (which see nothing)."""
    case = C.attend_case([40, 3, 0], [6, 9, 4], 4, 2, dim, 16, dtype, seed=21)
    if short:
        case["seq_lens"] = torch.tensor([40, 3, 0], dtype=torch.int32)
    g = C.on_gpu(case)
    args = [g[n] for n in ("q", "k_cache", "v_cache", "block_table", "seq_lens", "cu_tokens")]
    full = sv.kv_paged_attention(*args, lse=True)
    longest = int(case["seq_lens"].max())
    for window in (2 ** 31 - 1, 2 ** 31 - 2, 46, 45, 41, 40, 39):
        r = sv.kv_paged_attention(*args, lse=True, sliding_window=window)
        torch.cuda.synchronize()
        same = torch.equal(r["out"], full["out"]) and torch.equal(r["lse"], full["lse"])
        assert same == (window >= longest), window
        C.check(C.to64(r["out"]), C.to64(r["lse"]), C.reference(case, window=window), dtype, dim)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_token_ranges_that_overlap_touch_nothing_else(sv, dtype):
    """Offsets that do not ascend can ask for more tiles than were launched: none
    is computed then, and the outputs keep their values."""
    B, n = 12, 160
    g = C.on_gpu(C.attend_case([500] * B, [n] + [0] * (B - 1), 4, 2, 128, 16, dtype, seed=22))
    cu = torch.tensor([0, n] * (B // 2) + [0], dtype=torch.int32, device=C.DEV)
    args = [g[k] for k in ("q", "k_cache", "v_cache", "block_table", "seq_lens")]
    guard = torch.full((n + 8, 4, 128), 3.0, dtype=g["q"].dtype, device=C.DEV)
    r = sv.kv_paged_attention(*args, cu, max_new=n,
                              out=dict(out=guard[4:n + 4], lse=None, workspace=None))
    torch.cuda.synchronize()
    assert r["out"].shape[0] == n and (guard == 3.0).all()


def test_two_graphs_share_a_workspace(sv):
    """Two captured calls of different shapes on one workspace, replayed in turn."""
    names = ("q", "k_cache", "v_cache", "block_table", "seq_lens", "cu_tokens")
    cases = [C.on_gpu(C.attend_case([6000, 30], [5, 9], 8, 2, 128, 16, "bf16", seed=23)),
             C.on_gpu(C.attend_case([2500, 900, 7], [1, 1, 1], 4, 4, 64, 8, "f16", seed=24))]
    alone = [sv.kv_paged_attention(*[c[n] for n in names]) for c in cases]
    torch.cuda.synchronize()
    shared = max((r["workspace"] for r in alone), key=lambda w: w.numel())
    outs = [dict(out=torch.zeros_like(r["out"]), lse=None, workspace=shared) for r in alone]
    graphs = []
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for c, o in zip(cases, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.stream(s):
            with torch.cuda.graph(graphs[-1], stream=s):
                sv.kv_paged_attention(*[c[n] for n in names], out=o)
    for rep in range(6):
        for o in outs:
            o["out"].fill_(2.0)
        torch.cuda.synchronize()
        graphs[rep % 2].replay()
        graphs[1 - rep % 2].replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, alone):
            assert torch.equal(o["out"], r["out"])


@pytest.mark.parametrize("dim", [8, 24, 40, 56, 72, 80, 96, 120, 136, 160, 192, 248])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_head_sizes_between(sv, dtype, dim):
    """Head sizes that fill a part of the matrix kernel's rows: every tile height,
    with split keys and without, windows, neighbouring memory of NaN."""
    for i, (ctx, new, heads, kv, bs, window) in enumerate([
            ([3000, 5], [1, 1], 4, 2, 16, 0), ([70, 400], [9, 20], 2, 2, 24, 0),
            ([33, 0, 600], [40, 7, 50], 3, 3, 5, 100), ([10, 700], [150, 60], 4, 2, 32, 0),
            ([2500], [130], 2, 1, 16, 0)]):
        case = C.attend_case(ctx, new, heads, kv, dim, bs, dtype, seed=40 + i, lead=2, tail=3,
                             fused=i % 2 == 1)
        g = C.on_gpu(case)
        T = case["q"].shape[0]
        guard = torch.full((T + 2, heads, dim), 7.0, dtype=C.DT[dtype], device=C.DEV)
        lse = torch.full((T, heads), 7.0, device=C.DEV)
        sv.kv_paged_attention(*[g[n] for n in ("q", "k_cache", "v_cache", "block_table",
                                               "seq_lens", "cu_tokens")], sliding_window=window,
                              max_new=max(new),
                              out=dict(out=guard[1:T + 1], lse=lse, workspace=None))
        torch.cuda.synchronize()
        C.check(C.to64(guard[1:T + 1]), C.to64(lse), C.reference(case, window=window), dtype, dim,
                (i, dim))
        assert (guard[:3] == 7.0).all() and (guard[-4:] == 7.0).all() and (lse[-3:] == 7.0).all()
