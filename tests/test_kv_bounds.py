"""The bounds of tests/kvbounds.py on the CPU: over long contexts they take what the
kernels' arithmetic gives and refuse outputs that are wrong -- zeros, the sign,
a part of the keys left out, another head's values -- in every type."""

import numpy as np
import pytest
import torch

from tests import kvbounds as B
from tests import kvcases as C

LONG = [([9001, 10], 1, 64), ([9001, 4000], 3, 128), ([2500, 10], 40, 72), ([3000], 1, 80),
        ([700], 60, 256)]


def _kernel_like(case, ref, dtype):
    """Attention with scores and weights in float32, the weights rounded to the type
    before the product as the 16-bit kernels do (their largest is 2^7 in float16)."""
    out = np.zeros_like(ref["out"])
    q = case["q"].float()
    T, H, D = q.shape
    kv, bs = case["k_cache"].shape[1], case["k_cache"].shape[2]
    cu, lens = case["cu_tokens"].tolist(), case["seq_lens"].tolist()
    for b, L in enumerate(lens):
        pos = torch.arange(L)
        page = case["block_table"][b, pos // bs].long()
        for h in range(H):
            k = case["k_cache"][page, h * kv // H, pos % bs].float()
            v = case["v_cache"][page, h * kv // H, pos % bs].float()
            for t in range(cu[b], cu[b + 1]):
                p = L - cu[b + 1] + t
                s = (k[:p + 1] @ q[t, h]) * D ** -0.5
                w = torch.exp(s - s.max()) * (128.0 if dtype == "f16" else 1.0)
                o = (w.to(C.DT[dtype]).float() @ v[:p + 1]) / w.sum()
                out[t, h] = C.to64(o.to(C.DT[dtype]))
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ctx,new,dim", LONG, ids=lambda x: str(x).replace(" ", ""))
def test_wrong_outputs_are_refused(dtype, ctx, new, dim):
    case = C.attend_case(ctx, [new] * len(ctx), 2, 1, dim, 16, dtype, seed=new)
    ref = C.reference(case)
    right = _kernel_like(case, ref, dtype)
    assert B.check(right, ref["lse"], ref, dtype, dim) <= 1.0
    # the sequence of the longest context alone is wrong
    rows = slice(0, new)
    less = {**case, "block_table": case["block_table"].clone()}
    less["block_table"][0, 8:40] = -1                 # 512 positions left out
    heads = right[:, ::-1].copy()
    for name, wrong in (("zeros", np.zeros_like(right)), ("sign", -right), ("heads", heads),
                        ("keys", C.reference(less)["out"])):
        bad = right.copy()
        bad[rows] = wrong[rows]
        with pytest.raises(AssertionError):
            B.check(bad, ref["lse"], ref, dtype, dim, name)
