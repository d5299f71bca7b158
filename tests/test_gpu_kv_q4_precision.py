"""How much of its operands kv_paged_attention_q4 keeps, in calls whose results are
known in closed form."""

import math

import numpy as np
import pytest
import torch

from tests import kvcases as C
from tests import kvq4cases as Q

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_token_verification_amd as m
    m.library()
    return m


def _one_channel_keys(dim, kv, byte):
    """A sequence of ``dim`` tokens, the key of the t-th with 6 * 2^(byte - 127) in channel
    t and 0 elsewhere, in pages that lie backwards."""
    n = dim // 16
    c = dict(k_codes=torch.zeros((n, kv, 16, dim // 2), dtype=torch.uint8),
             k_scales=torch.full((n, kv, 16, -(-dim // 128) * 4), byte, dtype=torch.uint8),
             v_codes=torch.full((n, kv, 16, dim // 2), 0x22, dtype=torch.uint8),
             v_scales=torch.ones((n, kv, 16)))
    t = torch.arange(dim)
    for h in range(kv):
        c["k_codes"][n - 1 - t // 16, h, t % 16, t // 2] = torch.where(t % 2 == 0, 0x07, 0x70).to(torch.uint8)
    return c, torch.arange(n - 1, -1, -1, dtype=torch.int32)[None]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("byte,scale", [(127, 1.0), (127, None), (129, 0.013), (245, 2.0 ** -120),
                                        (20, 2.0 ** 107)])
def test_scores_hold_queries_whole(sv, byte, scale, dim, dtype):
    """Every token sees itself alone, so its lse is scale * 6 * 2^(byte - 127) times one
    channel of its query, x.

    Channels of a 128th (bfloat16; float16: of a 512th) of the largest of their 32 are
    held whole, so the product, of 8 or 11 bits times 6, is exact in float32.  In log2
    units, with y = |lse| log2 e and steps of u = 2^-24 relative: the factor scale * log2
    e is off by 2 u and the reference's product by u, y each; the reference, 8 more, by
    (y + 8) u; the weight's exponent by (8 + 3 y u) u and 3 y u, and by 4 u the
    exponential; the logarithm (of 2^-8) by 16 u, the sum by y u.  The last product is
    off by 2 u.  All in all less than 12 u y + 64 u."""
    heads, kv = 4, 2
    g = torch.Generator().manual_seed(dim)
    cache, table = _one_channel_keys(dim, kv, byte)
    low = -7.0 if dtype == "bf16" else -9.0
    x = torch.exp2(torch.rand((dim, heads, dim), generator=g) * low)
    x = x.view(dim, heads, dim // 32, 32)
    x[..., 5] = 1.999                              # the largest
    x = (x.clamp(min=2.0 ** (low + 1)) * (2 * torch.randint(0, 2, x.shape, generator=g) - 1))
    case = dict(q=x.view(dim, heads, dim).to(C.DT[dtype]), cache=cache, block_table=table,
                seq_lens=torch.tensor([dim], dtype=torch.int32),
                cu_tokens=torch.tensor([0, dim], dtype=torch.int32))
    gpu = Q.on_gpu(case)
    r = sv.kv_paged_attention_q4(*[gpu[n] for n in Q.NAMES], lse=True, scale=scale, sliding_window=1)
    torch.cuda.synchronize()
    at = np.arange(dim)
    s = float(np.float32(dim ** -0.5 if scale is None else scale))
    want = s * 6.0 * 2.0 ** (byte - 127) * C.to64(case["q"])[at, :, at]
    off = np.abs(C.to64(r["lse"]) - want)
    bound = (12 * np.abs(want) / math.log(2) + 64) * U
    print(f"{(off / bound).max():.3f} of the bound")
    assert (off <= bound).all(), (off / bound).max()
    assert (C.to64(r["out"]) == 1.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [32, 64, 128, 224, 256])
@pytest.mark.parametrize("steps", [9.0, 10.95, 13.0])
def test_many_weights_far_below_one(sv, steps, dim, dtype):
    """A token over 128 or 640 positions with one key in 32 that outweighs each of the
    others by 2^steps; all values are 6 units.  The others' share stays in the output as
    in the sum of the weights: the output is 6 units.

    A weight times its scale is off by 2^-14 of the largest of its lane's 32 at most, a
    lane's 32 by 2^-9 of it, and the sum of the weights is not less than that largest.  The
    rest of it is float32 (640 sums and some steps of 2^-24, and the exponential's), the
    output is rounded once."""
    half = torch.finfo(C.DT[dtype]).eps / 2
    for L in (128, 640):
        n, heads = L // 16, 4
        unit = 0.9453125                  # times a weight of a power of two just over 3.75 / 4
        c = dict(k_codes=torch.zeros((n, 1, 16, dim // 2), dtype=torch.uint8),
                 k_scales=torch.full((n, 1, 16, -(-dim // 128) * 4), 127, dtype=torch.uint8),
                 v_codes=torch.full((n, 1, 16, dim // 2), 0x77, dtype=torch.uint8),
                 v_scales=torch.full((n, 1, 16), unit))
        c["k_codes"][0::8, 0, 0::4, 0] = 0x07     # of each lane's 32 of 128 positions the first
        q = torch.zeros((1, heads, dim), dtype=C.DT[dtype])
        q[:, :, 0] = 1.0
        case = dict(q=q, cache=c, block_table=torch.arange(n, dtype=torch.int32)[None],
                    seq_lens=torch.tensor([L], dtype=torch.int32),
                    cu_tokens=torch.tensor([0, 1], dtype=torch.int32))
        gpu = Q.on_gpu(case)
        r = sv.kv_paged_attention_q4(*[gpu[m] for m in Q.NAMES], lse=True,
                                     scale=steps * math.log(2) / 6)
        torch.cuda.synchronize()
        off = (np.abs(C.to64(r["out"]) / (6 * unit) - 1)).max()
        bound = 2.0 ** -9 + half * (1 + 2.0 ** -9) + 700 * U
        print(f"{L}: {off:.2e}, {off / bound:.3f} of the bound")
        assert off <= bound, (L, off, bound)
        lse = steps * math.log(2) + math.log((L // 32) * (1 + 31 * 2.0 ** -steps))
        assert np.abs(C.to64(r["lse"]) - lse).max() <= (L + 80) * U * 12


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,ctx,new,heads,kv", [
    (64, [700, 30], [3, 40], 8, 2), (128, [1500, 0], [9, 100], 8, 2), (256, [300, 1], [5, 33], 4, 4),
    (96, [2500], [1], 6, 2)])
def test_outputs_within_three_pieces(sv, dim, ctx, new, heads, kv, dtype):
    """The bounds of tests/kvq4cases.py with 2^-14 of the largest of a lane's 32 positions
    for the weights of either type."""
    case = Q.attend_case(ctx, new, heads, kv, dim, 16, dtype, seed=70)
    gpu = Q.on_gpu(case)
    r = sv.kv_paged_attention_q4(*[gpu[m] for m in Q.NAMES], lse=True)
    torch.cuda.synchronize()
    ref = Q.reference(case)
    half = torch.finfo(C.DT[dtype]).eps / 2
    e_s = 2.0 ** (-14 if dtype == "bf16" else -19) * ref["split_abs"] + \
        (dim + 8) * U * (2.1 * ref["score_abs"] + 8 * math.log(2))
    rel = 2 * np.expm1(2 * e_s + 24 * U)[..., None] + (ref["keys"][..., None] + 16) * U
    tol = rel * ref["weight_abs"] + 2.0 ** -14 * (1 + rel) * ref["piece_abs"]
    tol = tol * 1.01 + half * (np.abs(ref["out"]) + tol) + 2.0 ** -25
    off = np.abs(C.to64(r["out"]) - ref["out"])
    rounded = np.abs(torch.from_numpy(ref["out"]).to(C.DT[dtype]).double().numpy() - ref["out"])
    print(f"{(off / tol).max():.3f} of the bound, {np.sqrt((off ** 2).sum() / (rounded ** 2).sum()):.3f} "
          "times the rounding alone")
    assert (off <= tol).all(), (off / tol).max()
