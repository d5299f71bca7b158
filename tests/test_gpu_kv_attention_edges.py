"""GPU parity of kv_paged_attention at calls that its other tests leave out, within
bounds by arithmetic (tests/kvcases.py, tests/kvbounds.py)."""

import numpy as np
import pytest
import torch

from tests import kvbounds as B
from tests import kvcases as C

pytestmark = pytest.mark.gpu

NAMES = ("q", "k_cache", "v_cache", "block_table", "seq_lens", "cu_tokens")


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_token_verification_amd as m
    m.library()
    return m


@pytest.mark.parametrize("ctx,new,heads,dim,dtype,hint", [
    (60, 140, 256, 64, "bf16", 1),       # 5 tiles of 32 rows for 4 places a head
    (10, 200, 128, 128, "f16", 1),       # 7 for 6
    (70, 160, 64, 64, "f32", 0),         # 40 tiles of 4 rows for 16
    (1, 40, 128, 248, "f32", 0),         # 20 of 2 for 4
    (9, 150, 256, 256, "bf16", 0)])      # 3 tiles of 64 rows for 2
def test_one_sequence_of_more_tiles_than_places(sv, ctx, new, heads, dim, dtype, hint):
    """A single sequence whose tiles alone fill the chip, on a table so wide that its
    keys could be split."""
    case = C.attend_case([ctx], [new], heads, heads, dim, 16, dtype, seed=31)
    wide = torch.full((1, 600), -1, dtype=torch.int32)
    wide[:, :case["block_table"].shape[1]] = case["block_table"]
    g = C.on_gpu({**case, "block_table": wide})
    r = sv.kv_paged_attention(*[g[n] for n in NAMES], lse=True, max_new=hint)
    torch.cuda.synchronize()
    assert r["workspace"] is not None
    C.check(C.to64(r["out"]), C.to64(r["lse"]), C.reference(case), dtype, dim)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("gap", [12.75, 16.90625, 17.40625])
@pytest.mark.parametrize("dim,heads,kv", [(64, 32, 8), (128, 16, 4), (256, 8, 8)])
def test_flat_tail_behind_a_dominant_key(sv, dtype, gap, dim, heads, kv):
    """Every key but the first scores ``gap`` (in the type) below it (18.4 to 25.1 in log2 units):
    the output is the tail's share, p w / (1 + p w) at position p, w = exp(-gap)."""
    T, bs = 4096 if dtype != "f32" else 700, 16
    dt = C.DT[dtype]
    g = torch.Generator().manual_seed(int(gap * 32) + dim)
    table = torch.randperm(T // bs + 1, generator=g).to(torch.int32)[None].to(C.DEV)
    k = torch.zeros((T // bs + 1, kv, bs, dim), dtype=dt, device=C.DEV)
    v = torch.ones_like(k)
    k[table[0, 0].item(), :, 0, 1] = gap
    gap = float(k[table[0, 0].item(), 0, 0, 1])     # as the type holds it
    v[table[0, 0].item(), :, 0] = 0.0
    q = torch.zeros((T, heads, dim), dtype=dt, device=C.DEV)
    q[:, :, 1] = 1.0
    r = sv.kv_paged_attention(q, k, v, table, torch.tensor([T], dtype=torch.int32, device=C.DEV),
                              torch.tensor([0, T], dtype=torch.int32, device=C.DEV), scale=1.0,
                              lse=True, max_new=T)
    torch.cuda.synchronize()
    p = np.arange(T)[:, None]
    tail = np.broadcast_to(p * np.exp(-gap), (T, heads))
    ref = dict(out=np.broadcast_to((tail / (1 + tail))[..., None], (T, heads, dim)),
               lse=gap + np.log1p(tail), keys=np.broadcast_to(p + 1.0, (T, heads)),
               v_max=np.ones((T, heads)), score_abs=np.full((T, heads), gap),
               score_top=np.full((T, heads), gap))
    ref["weight_abs"] = ref["out"]
    share = B.check(C.to64(r["out"]), C.to64(r["lse"]), ref, dtype, dim)
    print(f"{share:.3f} of the bound")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ctx,new", [([100], [1]), ([6000, 40], [2, 40])])
def test_values_near_the_largest(sv, dtype, dim, ctx, new):
    """Values of 4e36: a late key that outweighs the ones before it by 2^7.5 leaves the
    sums finite."""
    case = C.attend_case(ctx, new, 2, 1, dim, 16, dtype, seed=33)
    case["q"].zero_()
    case["q"][:, :, 0] = 1.0
    for b, L in enumerate(case["seq_lens"].tolist()):
        pos = torch.arange(L)
        page, at = case["block_table"][b, pos // 16].long(), pos % 16
        case["k_cache"][page, 0, at] = 0.0
        last = (ctx[b] - 1) // 16, (ctx[b] - 1) % 16
        case["k_cache"][case["block_table"][b, last[0]].long(), 0, last[1], 0] = 5.1875
        case["v_cache"][page, 0, at] *= 4e36
    g = C.on_gpu(case)
    r = sv.kv_paged_attention(*[g[n] for n in NAMES], scale=1.0, lse=True)
    torch.cuda.synchronize()
    B.check(C.to64(r["out"]), C.to64(r["lse"]), C.reference(case, 1.0), dtype, dim)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256, 72])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_long_contexts(sv, dtype, dim, new):
    """Split keys and their joining within bounds that are sharp over long contexts."""
    ctx = [2500, 10] if new == 40 and dim > 64 else [9001, 10, 4000]
    case = C.attend_case(ctx, [new] * len(ctx), 2, 1, dim, 16, dtype, seed=50 + new)
    g = C.on_gpu(case)
    r = sv.kv_paged_attention(*[g[n] for n in NAMES], lse=True)
    torch.cuda.synchronize()
    share = B.check(C.to64(r["out"]), C.to64(r["lse"]), C.reference(case), dtype, dim)
    print(f"{share:.3f} of the bound")


@pytest.mark.parametrize("dim", [8, 24, 40, 56, 72, 80, 96, 120, 136, 160, 192, 248])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_long_contexts_of_head_sizes_between(sv, dtype, dim):
    for i, (ctx, new, heads, kv, bs, window) in enumerate([
            ([3000, 5], [1, 1], 4, 2, 16, 0), ([70, 400], [9, 20], 2, 2, 24, 0),
            ([10, 700], [150, 60], 4, 2, 32, 0), ([2500], [130], 2, 1, 16, 0)]):
        case = C.attend_case(ctx, new, heads, kv, dim, bs, dtype, seed=60 + i)
        g = C.on_gpu(case)
        r = sv.kv_paged_attention(*[g[n] for n in NAMES], lse=True, max_new=max(new))
        torch.cuda.synchronize()
        B.check(C.to64(r["out"]), C.to64(r["lse"]), C.reference(case), dtype, dim, (i, dim))


def test_reused_outputs_take_any_hint_and_window(sv):
    """One out dict over calls whose hint and window ask for larger workspaces, in any
    order; a call captured with the first workspace still replays right."""
    case = C.attend_case([9000, 5000, 40, 7], [10, 10, 10, 10], 32, 8, 128, 16, "bf16", seed=34)
    g = C.on_gpu(case)
    args = [g[n] for n in NAMES]
    out = sv.kv_paged_attention(*args, max_new=1)
    first = out["workspace"]
    alone = out["out"].clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            sv.kv_paged_attention(*args, max_new=1, out=out)
    del first
    grown = set()
    for hint, window in ((1, 0), (9, 0), (40, 0), (1, 512), (9, 512), (40, 300), (0, 0), (9, 0)):
        fresh = sv.kv_paged_attention(*args, max_new=hint, sliding_window=window)
        r = sv.kv_paged_attention(*args, max_new=hint, sliding_window=window, out=out)
        torch.cuda.synchronize()
        assert r is out and torch.equal(r["out"], fresh["out"]), (hint, window)
        grown.add(r["workspace"].numel())
        # memory that the allocator hands out again is not the captured call's
        junk = [torch.full((n,), 0x7f, dtype=torch.uint8, device=C.DEV) for n in sorted(grown)]
        out["out"].fill_(1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["out"], alone), (hint, window)
        assert all((j == 0x7f).all() for j in junk)
        del junk
    assert len(grown) > 1
    # an explicit workspace is the caller's
    small = torch.empty(min(grown) - 256, dtype=torch.uint8, device=C.DEV)
    with pytest.raises(sv.SpecVerifyError, match="workspace has"):
        sv.kv_paged_attention(*args, max_new=1, out=out, workspace=small)


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("f16", 128), ("f32", 64)])
def test_batches_of_thousands(sv, dtype, dim):
    """Single tokens and short windows of 5000 sequences, one long one among them."""
    rng = np.random.default_rng(35)
    ctx, new = rng.integers(0, 30, 5000).tolist(), rng.integers(0, 3, 5000).tolist()
    ctx[4321], new[4321] = 3000, 2
    case = C.attend_case(ctx, new, 2, 1, dim, 16, dtype, seed=35)
    g = C.on_gpu(case)
    r = sv.kv_paged_attention(*[g[n] for n in NAMES], lse=True, max_new=2)
    torch.cuda.synchronize()
    B.check(C.to64(r["out"]), C.to64(r["lse"]), C.reference(case), dtype, dim)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scores_of_minus_infinity_alone_give_zero(sv, dtype, dim, bad):
    """Whatever the values there hold, with split keys and without."""
    for ctx, new in (([40, 6000, 30], [3, 1, 20]), ([300], [70])):
        case = C.attend_case(ctx, new, 2, 1, dim, 16, dtype, seed=37)
        case["q"].zero_()
        case["q"][:, :, 3] = 1.0
        L = int(case["seq_lens"][-1 if len(ctx) == 1 else 1])
        b = len(ctx) // 2
        pos = torch.arange(L)
        page = case["block_table"][b, pos // 16].long()
        case["k_cache"][page, 0, pos % 16, 3] = float("-inf")
        clean = {**case, "k_cache": case["k_cache"].clone(), "v_cache": case["v_cache"].clone()}
        clean["k_cache"][page, 0, pos % 16, 3] = 0.0
        case["v_cache"][page[::7], 0, pos[::7] % 16, 1] = bad
        g = C.on_gpu(case)
        r = sv.kv_paged_attention(*[g[n] for n in NAMES], lse=True)
        torch.cuda.synchronize()
        rows = slice(int(case["cu_tokens"][b]), int(case["cu_tokens"][b + 1]))
        assert (r["out"][rows] == 0).all() and torch.isneginf(r["lse"][rows]).all(), (ctx, new)
        ref = C.reference(clean)
        ref["lse"][rows] = np.nan                # checked above
        B.check(C.to64(r["out"]), C.to64(r["lse"]), ref, dtype, dim)
