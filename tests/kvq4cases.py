"""Inputs, references and error bounds shared by the tests of the 4-bit cache."""

import math

import numpy as np
import torch

from oracle import kvq4
from tests import kvcases as C

DEV = C.DEV
CACHE = ("k_codes", "k_scales", "v_codes", "v_scales")
NAMES = ("q", "cache", "block_table", "seq_lens", "cu_tokens")


def quantised(k, v):
    """The four arrays of float32 rows [.., dim], by torch on the CPU (checked against the
    oracle, code by code, in test_oracle_kvq4)."""
    dim = k.shape[-1]
    groups = k.reshape(*k.shape[:-1], dim // 32, 32).double()
    byte = torch.zeros(groups.shape[:-1], dtype=torch.int64)
    top = groups.abs().amax(-1)
    e = torch.ceil(torch.log2(top / 7)).nan_to_num(-127, 128, -127).clamp(-127, 127)
    e = torch.where(top > 7 * torch.exp2(e), e + 1, e)
    e = torch.where((top <= 3.5 * torch.exp2(e)) & (e > -127), e - 1, e)
    byte = torch.where(torch.isfinite(top), e + 127, 255).to(torch.uint8)
    unit = torch.exp2(e)
    unit_v = (v.abs().amax(-1).double() / 6).float().bfloat16().float()
    unit_v = torch.where(torch.isfinite(v).all(-1), unit_v, math.nan)
    kc, vc = _codes(groups / unit[..., None]).reshape(k.shape), _codes(
        v.double() / torch.where(unit_v > 0, unit_v, math.inf).double()[..., None])
    scales = torch.zeros((*k.shape[:-1], -(-dim // 128) * 4), dtype=torch.uint8)
    scales[..., :dim // 32] = byte
    return dict(k_codes=_packed(kc), k_scales=scales, v_codes=_packed(vc), v_scales=unit_v)


def _codes(x):
    level = torch.tensor(kvq4.MAGNITUDES, dtype=torch.float64)
    gap = (x.abs()[..., None].clamp(max=6.0) - level).abs()
    # (of two equally near the first with an even code)
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7])
    pick = order[gap[..., order].argmin(-1)]
    return torch.where(torch.isfinite(x), pick | torch.signbit(x).long() * 8, 0).to(torch.uint8)


def _packed(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def attend_case(ctx, new, heads, kv, dim, bs, dtype, seed=0, poison=True, lead=0, tail=0, spare=3,
                q_std=1.0, fused=False, k_std=1.0):
    """A case of C.attend_case with its caches in 4 bits.  Slots that no sequence holds
    have random codes, units that are NaN or large, scales that are NaN or infinite."""
    case = C.attend_case(ctx, new, heads, kv, dim, bs, "f32", seed, 0.0, lead, tail, spare, q_std)
    g = torch.Generator().manual_seed(seed + 1000)
    k, v = case.pop("k_cache") * k_std, case.pop("v_cache")
    cache = quantised(k, v)
    if poison:
        held = torch.zeros((k.shape[0], bs), dtype=torch.bool)
        for b, L in enumerate(case["seq_lens"].tolist()):
            pos = torch.arange(L)
            held[case["block_table"][b, pos // bs].long(), pos % bs] = True
        bad = ~held[:, None].expand(-1, kv, -1)
        for n in ("k_codes", "v_codes"):
            noise = torch.randint(0, 256, cache[n].shape, generator=g, dtype=torch.uint8)
            cache[n] = torch.where(bad[..., None], noise, cache[n])
        odd = torch.tensor([255, 254, 200, 0], dtype=torch.uint8)[
            torch.randint(0, 4, cache["k_scales"].shape, generator=g)]
        cache["k_scales"] = torch.where(bad[..., None], odd, cache["k_scales"])
        odd = torch.tensor([math.nan, math.inf, 3e38, -1.0])[torch.randint(0, 4, bad.shape, generator=g)]
        cache["v_scales"] = torch.where(bad, odd, cache["v_scales"])
        # bytes that no channel uses
        cache["k_scales"][..., dim // 32:] = 255
    case["cache"] = {n: t.contiguous() for n, t in cache.items()}
    T = case["q"].shape[0]
    wide = torch.zeros((T, heads * dim + (24 if fused else 0)), dtype=C.DT[dtype])
    wide[:, :heads * dim] = case["q"].reshape(T, -1).to(C.DT[dtype])
    q = wide[:, :heads * dim].view(T, heads, dim)
    case["q"] = q if fused else q.contiguous()
    return case


def on_gpu(case):
    out = C.on_gpu({n: t for n, t in case.items() if n != "cache"})
    out["cache"] = {n: t.to(DEV) for n, t in case["cache"].items()}
    return out


def reference(case, scale=None, window=0):
    """float64 attention over what the codes stand for, and what its error bounds
    need: as ``oracle.pagedkv.paged_attention``, with split_abs [T, H] the largest
    scale * sum over 32 channels of max|q| * |k| (per unit of the split's error) and
    piece_abs [T, H, D] the sum over a lane's 32 positions of the largest weight
    times its scale, times the sum of the levels' magnitudes."""
    q = C.to64(case["q"])
    T, H, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    c = {n: t.numpy() for n, t in case["cache"].items()}
    table, lens, cu = (case[n].numpy() for n in ("block_table", "seq_lens", "cu_tokens"))
    nb, kv, bs, _ = c["k_codes"].shape
    group = H // kv
    r = dict(out=np.full((T, H, D), np.nan), lse=np.full((T, H), np.nan),
             weight_abs=np.zeros((T, H, D)), score_abs=np.zeros((T, H)), keys=np.zeros((T, H)),
             split_abs=np.zeros((T, H)), piece_abs=np.zeros((T, H, D)))
    for b in range(len(lens)):
        t0, t1, L = int(cu[b]), int(cu[b + 1]), int(lens[b])
        ends = min(max(L, 0), table.shape[1] * bs)
        s = np.array([i for i in range(ends) if 0 <= table[b, i // bs] < nb], dtype=np.int64)
        page, at = table[b, s // bs], s % bs
        for h in range(kv):
            k = kvq4.key_values(c["k_codes"][page, h, at], c["k_scales"][page, h, at]).reshape(-1, D)
            level = kvq4.unpack(c["v_codes"][page, h, at]).reshape(-1, D)
            unit = c["v_scales"][page, h, at].astype(np.float64)
            block = s // 128 * 4 + s % 16 // 4
            for t in range(t0, t1):
                p = L - (t1 - t0) + (t - t0)
                see = (s <= p) & ((s > p - window) if window else True)
                for e in range(h * group, (h + 1) * group):
                    if not see.any():
                        r["out"][t, e], r["lse"][t, e] = 0.0, -np.inf
                        continue
                    x = scale * (k[see] @ q[t, e])
                    m = x.max()
                    w = np.exp(x - m)
                    z = w.sum()
                    v = level[see] * unit[see, None]
                    r["out"][t, e] = w @ v / z
                    r["lse"][t, e] = m + np.log(z)
                    r["weight_abs"][t, e] = w @ np.abs(v) / z
                    r["score_abs"][t, e] = scale * (np.abs(k[see]) @ np.abs(q[t, e])).max()
                    r["keys"][t, e] = see.sum()
                    top = np.repeat(np.abs(q[t, e]).reshape(-1, 32).max(1), 32)
                    r["split_abs"][t, e] = scale * (np.abs(k[see]) @ top).max()
                    ids, inv = np.unique(block[see], return_inverse=True)
                    big = np.zeros(len(ids))
                    np.maximum.at(big, inv, w * unit[see])
                    sums = np.zeros((len(ids), D))
                    np.add.at(sums, inv, np.abs(level[see]))
                    r["piece_abs"][t, e] = big @ sums / z
    return r


def bounds(ref, dtype, dim):
    """Error bounds of out [T, H, D] and lse [T, H] by arithmetic.

    A query is off by 2^-14 (bfloat16; 2^-19 float16) of the largest of its 32
    channels, so a score by that times split_abs.  Its float32 sum starts from the
    row's reference, which is within 8 log2 units of a score, and takes dim products
    in up to 4 pieces whose magnitudes add up to 1.1 of the score's: every partial sum
    is below 2.1 score_abs + 8 ln 2, and dim + 8 of them round by 2^-24 each.  A
    weight is relatively off by twice the error of a score (its own and the
    largest's), the exponential's steps and the reference's rounding (within 16 log2
    units).

    A weight times its scale, x, in two pieces (bfloat16) over a unit s, where the
    largest of its lane's 32 positions is in (3.75 s, 7.5 s].  A piece's step is s / 2
    from 4 s on, s / 4 from 2 s on, s / 8 below that.  x of 4 s or more leaves s / 4 at
    most, 8 units of the second piece, which ends at 7.5: off by half of one of these,
    s / 64 <= 2^-8 x.  x in [2 s, 4 s) leaves s / 8, 4 of them, and is off by an eighth
    of one, s / 256 <= 2^-9 x; below that it leaves s / 16, 2 of them, off by a
    sixteenth, s / 512, which is 2^-10.9 of the largest at most.  Three pieces
    (float16), the largest in [2 s, 4 s): 2^-14 of it.  Float32 sums over n keys add
    n 2^-24 relative to the absolute sum, joins and the division 16 steps; the output
    is rounded once to its type."""
    half = torch.finfo(C.DT[dtype]).eps / 2
    split = 2.0 ** (-14 if dtype == "bf16" else -19)
    own, piece = (2.0 ** -8, 2.0 ** -9 / 3.75) if dtype == "bf16" else (0.0, 2.0 ** -14)
    u = 2.0 ** -24
    n = ref["keys"][..., None]
    e_s = split * ref["split_abs"] + (dim + 8) * u * (2.1 * ref["score_abs"] + 8 * math.log(2))
    e_w = 2 * e_s + 24 * u
    rel = 2 * np.expm1(e_w)[..., None] + (n + 16) * u
    tol = (rel + own * (1 + rel)) * ref["weight_abs"] + piece * (1 + rel) * ref["piece_abs"]
    tol = tol * 1.01 + half * (np.abs(ref["out"]) + tol)
    if dtype == "f16":
        tol = tol + 2.0 ** -25          # subnormal outputs
    lse = e_w + (ref["keys"] + 16) * u + 4 * u * np.abs(np.where(np.isfinite(ref["lse"]),
                                                               ref["lse"], 0.0))
    return tol, lse


def check(out, lse, ref, dtype, dim, note=""):
    """As C.check, with the bounds above."""
    mine = ~np.isnan(ref["lse"])
    tol, ltol = bounds(ref, dtype, dim)
    err = np.abs(out - ref["out"])[mine]
    assert np.isfinite(out[mine]).all(), (note, "not finite")
    share = float((err / np.maximum(tol[mine], 1e-300)).max()) if err.size else 0.0
    assert share <= 1.0, (note, "out", share, float(err.max()))
    if lse is not None:
        none = np.isneginf(ref["lse"])
        assert np.array_equal(np.isneginf(lse) & mine, none), (note, "empty rows")
        some = mine & ~none
        d = np.abs(lse - np.where(np.isfinite(ref["lse"]), ref["lse"], 0.0))[some]
        s2 = float((d / ltol[some]).max()) if d.size else 0.0
        assert s2 <= 1.0, (note, "lse", s2, float(d.max()))
        share = max(share, s2)
    return share
