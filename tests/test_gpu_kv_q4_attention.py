"""GPU parity of kv_paged_attention_q4 with float64 attention over what the codes
stand for, within bounds by arithmetic (tests/kvq4cases.py).  Slots that no
sequence holds have NaN units and infinite scales, so what is read from a masked
place shows."""

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


def _run(sv, case, **kw):
    g = Q.on_gpu(case)
    r = sv.kv_paged_attention_q4(*[g[n] for n in Q.NAMES], lse=True, **kw)
    torch.cuda.synchronize()
    return r


def _parity(sv, case, dtype, scale=None, window=0, **kw):
    r = _run(sv, case, scale=scale, sliding_window=window, **kw)
    ref = Q.reference(case, scale, window)
    return Q.check(C.to64(r["out"]), C.to64(r["lse"]), ref, dtype, case["q"].shape[2])


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
    ([100], [6], 3, 3, 96, 16, 0),                       # other head sizes
    ([70, 9], [2, 20], 4, 2, 160, 16, 0),
    ([33], [5], 2, 1, 32, 16, 0),
    ([120], [7], 4, 1, 192, 16, 30),
    ([60, 2], [12, 5], 6, 2, 224, 9, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"c{s[0][0]}n{s[1][0]}h{s[2]}-{s[3]}"
                         f"d{s[4]}bs{s[5]}w{s[6]}")
def test_attention_parity(sv, shape, dtype):
    ctx, new, heads, kv, dim, bs, window = shape
    for seed in (1, 2):
        case = Q.attend_case(ctx, new, heads, kv, dim, bs, dtype, seed=seed, fused=seed == 2)
        share = _parity(sv, case, dtype, window=window)
        print(f"{dtype} {shape}: {share:.3f} of the bound")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256, 96])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_split_keys_parity(sv, dtype, dim, new):
    """Few rows and long contexts: the key axis is split over workgroups and joined,
    beside a short sequence that is not."""
    ctx = [2500, 10] if new == 40 and dim > 64 else [9001, 10, 4000]
    case = Q.attend_case(ctx, [new] * len(ctx), 2, 1, dim, 16, dtype, seed=new)
    _parity(sv, case, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_peaked_and_large_scores(sv, dtype):
    """Scores of several hundred: the running maximum moves by much, most weights
    vanish."""
    for seed, std in ((1, 30.0), (2, 100.0)):
        case = Q.attend_case([700, 20], [9, 40], 4, 2, 128, 16, dtype, seed=seed, q_std=std)
        _parity(sv, case, dtype)
    case = Q.attend_case([700, 20], [9, 40], 4, 2, 128, 16, dtype, seed=3)
    _parity(sv, case, dtype, scale=1e-6)
    _parity(sv, case, dtype, scale=2.0)


@pytest.mark.parametrize("hint", [1, 3, 5, 10, 14, 17, 60, 10 ** 6])
def test_every_tile_shape_is_right_for_every_batch(sv, hint):
    """max_new only picks the tile shape."""
    case = Q.attend_case([40, 0, 333, 7], [1, 50, 9, 130], 8, 2, 128, 16, "bf16", seed=5)
    _parity(sv, case, "bf16", max_new=hint)
    _parity(sv, case, "bf16", max_new=hint, window=23)
    case = Q.attend_case([40, 0, 333, 7], [1, 50, 9, 130], 6, 2, 64, 16, "f16", seed=6)
    _parity(sv, case, "f16", max_new=hint)
    case = Q.attend_case([40, 7], [20, 70], 3, 3, 256, 16, "bf16", seed=7)
    _parity(sv, case, "bf16", max_new=hint)
