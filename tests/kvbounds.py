"""Error bounds of the paged attention that long contexts leave sharp, in float16
too (tests/kvcases.py charges every float16 weight the largest loss of any)."""

import numpy as np
import torch

from tests import kvcases as C


def out_bound(ref, dtype, dim):
    """Error bound of out [T, H, D] by arithmetic.

    As in kvcases.bounds, with e_w the relative error of a float32 weight, to
    which the reference's own rounding (a score within 16 of the largest, in log2
    units) adds 16 * 2^-24.  bf16 and f16 round a weight by half a step relative
    to it.  In f16 a weight below 2^-14 is subnormal and is rounded by up to
    2^-25 instead; the largest weight of a row and split is 2^7 or more in
    that scale, so the loss is at most 2^-32 of the largest weight of the row,
    which is 1 where the weights sum to z = exp(lse - top)."""
    half = torch.finfo(C.DT[dtype]).eps / 2
    u = 2.0 ** -24
    n = ref["keys"][..., None]
    e_w = (2 * (dim + 4) * ref["score_abs"] + 20) * u
    rel = 2 * e_w[..., None] + (n + 16) * u
    tol = (rel + (0.0 if dtype == "f32" else half)) * ref["weight_abs"]
    if dtype == "f16":
        some = np.isfinite(ref["lse"])
        z = np.where(some, np.exp(np.where(some, ref["lse"] - ref["score_top"], 0.0)), 1.0)
        tol = tol + (n * 2.0 ** -32) * (ref["v_max"] / z)[..., None]
    tol = tol * 1.01 + half * (np.abs(ref["out"]) + tol)
    if dtype == "f16":
        tol = tol + 2.0 ** -25          # subnormal outputs
    return tol


def check(out, lse, ref, dtype, dim, note=""):
    """kvcases.check, and out against the bound above; returns the largest error as a
    share of that."""
    C.check(out, lse, ref, dtype, dim, note)
    mine = ~np.isnan(ref["lse"])
    share = np.abs(out - ref["out"])[mine] / np.maximum(out_bound(ref, dtype, dim)[mine], 1e-300)
    worst = float(share.max()) if share.size else 0.0
    assert worst <= 1.0, (note, "out", worst)
    return worst
