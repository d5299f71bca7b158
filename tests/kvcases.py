"""Inputs and error bounds shared by the GPU tests of the paged-KV calls."""

import numpy as np
import torch

from oracle import pagedkv

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def to64(t):
    return t.detach().cpu().double().numpy()


def attend_case(ctx, new, heads, kv, dim, bs, dtype, seed=0, poison=float("nan"), lead=0, tail=0,
                spare=3, q_std=1.0, fused=False):
    """Caches, tables and queries of sequences with ``ctx`` cached and ``new``
    new tokens, on the CPU.  Every slot that no sequence holds is ``poison``;
    ``lead`` / ``tail`` query rows before and behind the sequences belong to none.
    ``fused``: q is a part of wider rows, the caches of one allocation."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    lens = [c + n for c, n in zip(ctx, new)]
    need = [-(-L // bs) for L in lens]
    nb = sum(need) + spare
    width = max(need + [1]) + 1
    order = torch.randperm(nb, generator=g)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    both = torch.full((nb, 2, kv, bs, dim), poison, dtype=dt)
    at = 0
    for b, (L, m) in enumerate(zip(lens, need)):
        ids = order[at:at + m]
        at += m
        table[b, :m] = ids.to(torch.int32)
        pos = torch.arange(L)
        for i in (0, 1):
            rows = torch.randn((L, kv, dim), generator=g).to(dt)
            both[ids[pos // bs], i, :, pos % bs] = rows
    T = lead + sum(new) + tail
    wide = torch.randn((T, heads * dim + (24 if fused else 0)), generator=g) * q_std
    q = wide.to(dt)[:, :heads * dim].view(T, heads, dim)
    cu = np.concatenate([[lead], lead + np.cumsum(new)])
    k, v = both[:, 0], both[:, 1]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    return dict(q=q, k_cache=k, v_cache=v, block_table=table,
                seq_lens=torch.tensor(lens, dtype=torch.int32),
                cu_tokens=torch.tensor(cu, dtype=torch.int32))


def on_gpu(case):
    """The case's tensors on the GPU with their strides kept."""
    out = {}
    for n, t in case.items():
        base = t if t.is_contiguous() else t._base
        moved = base.to(DEV)
        out[n] = moved if t.is_contiguous() else moved.as_strided(t.size(), t.stride(),
                                                                  t.storage_offset())
    return out


def reference(case, scale=None, window=0):
    D = case["q"].shape[2]
    return pagedkv.paged_attention(to64(case["q"]), to64(case["k_cache"]), to64(case["v_cache"]),
                                   case["block_table"].numpy(), case["seq_lens"].numpy(),
                                   case["cu_tokens"].numpy(), D ** -0.5 if scale is None else scale,
                                   window)


def bounds(ref, dtype, dim):
    """Error bounds of out [T, H, D] and lse [T, H] by arithmetic.

    A score is a float32 sum of dim products: off by at most (dim + 2) 2^-24
    score_abs (products and sums each half a step, the scale two).  The
    exponent's argument is a difference of two such scores rounded once more
    relative to the largest |score|; with the exponential's own 2 steps every
    weight is relatively off by
        e_w = 2 (dim + 4) 2^-24 score_abs + 4 * 2^-24.
    Float32 sums over n keys add n 2^-24 relative to the absolute sum, the
    merges of splits and the division 16 more steps.  bf16 and f16 round each
    weight by half a step eps/2 for the product with v (the sum of the weights is
    not rounded); f16 weights below 2^-14 lose up to 2^-15 absolutely where
    subnormals are flushed, against a sum of weights of at least 1.  The output
    is rounded once to its type."""
    half = torch.finfo(DT[dtype]).eps / 2      # of a value rounded to the type
    u = 2.0 ** -24
    n = ref["keys"][..., None]
    e_w = (2 * (dim + 4) * ref["score_abs"] + 4) * u
    rel = 2 * e_w[..., None] + (n + 16) * u
    weight = 0.0 if dtype == "f32" else half
    a = ref["weight_abs"]
    tol = (rel + weight) * a
    if dtype == "f16":
        tol = tol + n * 2.0 ** -15 * ref["v_max"][..., None]
    tol = tol * 1.01 + half * (np.abs(ref["out"]) + tol)
    if dtype == "f16":
        tol = tol + 2.0 ** -25          # subnormal outputs
    lse = e_w + (ref["keys"] + 16) * u + 4 * u * np.abs(np.where(np.isfinite(ref["lse"]),
                                                               ref["lse"], 0.0))
    return tol, lse


def check(out, lse, ref, dtype, dim, note=""):
    """Compares out / lse (CPU float64 arrays) with the reference on every row of
    a sequence; returns the largest error as a share of its bound."""
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
