"""The paged-KV calls as a decoding loop uses them, around the LM-head
verification: extend the tables for the drafted window, write its keys and
values, attend, verify, roll back what was rejected, take the freed blocks
back.  A toy early-exit model drives it (random projections of token
embeddings); every step is checked against the oracle and a dense cache."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import pagedkv
from tests import kvcases as C

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import lossless_token_verification_amd as m
    m.library()
    return m


class Loop:
    """State of B sequences: tables, lengths, pool, caches, and a dense copy of
    every sequence's keys and values for the checks."""

    def __init__(self, sv, B, k, bs, dtype, seed, width=12, heads=4, kv=2, dim=64, vocab=256):
        g = torch.Generator().manual_seed(seed)
        self.sv, self.B, self.k, self.bs, self.g = sv, B, k, bs, g
        self.heads, self.kv, self.dim, self.vocab, self.dt = heads, kv, dim, vocab, C.DT[dtype]
        blocks = B * width // 2 + 4
        self.table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.free = torch.randperm(blocks, generator=g).to(torch.int32).to(DEV)
        self.count = torch.tensor([blocks], dtype=torch.int32, device=DEV)
        self.kc = torch.full((blocks, kv, bs, dim), float("nan"), dtype=self.dt, device=DEV)
        self.vc = self.kc.clone()
        self.dense = [[[], []] for _ in range(B)]
        self.freed = torch.full((B, 2), -1, dtype=torch.int32, device=DEV)
        self.num_freed = torch.zeros(B, dtype=torch.int32, device=DEV)
        H = heads * dim
        w = lambda *s: (torch.randn(s, generator=g) * s[0] ** -0.5).to(self.dt).to(DEV)  # noqa: E731
        self.embed, self.wqkv = w(vocab, H) * 10, w(H, H + 2 * kv * dim)
        self.head = torch.randn((vocab, H), generator=g).to(torch.bfloat16).to(DEV)

    def step(self, tokens, counts):
        """Appends counts[b] tokens per sequence and returns their attention
        output [T, heads * dim]; checks the attention against the dense copy."""
        sv, T = self.sv, sum(counts)
        new = torch.tensor(counts, dtype=torch.int32, device=DEV)
        r = sv.kv_blocktable_extend(self.table, self.lens, new, self.free, self.count, self.bs, T,
                                    freed_blocks=self.freed, num_freed=self.num_freed)
        self.lens, self.count = r["new_lens"], r["free_left"]
        self.num_freed.zero_()
        assert (r["num_taken"] >= 0).all()
        x = torch.matmul(self.embed[tokens], self.wqkv)
        H, kvd = self.heads * self.dim, self.kv * self.dim
        q = x[:, :H].view(T, self.heads, self.dim)
        k = x[:, H:H + kvd].view(T, self.kv, self.dim)
        v = x[:, H + kvd:].view(T, self.kv, self.dim)
        sv.kv_cache_append(k, v, r["slot_map"], self.kc, self.vc)
        a = sv.kv_paged_attention(q, self.kc, self.vc, self.table, self.lens, r["cu_tokens"],
                                  lse=True, max_new=max(counts))
        torch.cuda.synchronize()
        at = 0
        for b, n in enumerate(counts):
            self.dense[b][0] += list(k[at:at + n].cpu())
            self.dense[b][1] += list(v[at:at + n].cpu())
            at += n
        self.check(q, a, counts)
        return a["out"].reshape(T, H)

    def check(self, q, a, counts):
        lens = [len(d[0]) for d in self.dense]
        assert self.lens.tolist() == lens
        width = max(lens + [1])
        kc = np.zeros((self.B, self.kv, width, self.dim))
        vc = np.zeros_like(kc)
        for b, (ks, vs) in enumerate(self.dense):
            if ks:
                kc[b, :, :len(ks)] = C.to64(torch.stack(ks)).transpose(1, 0, 2)
                vc[b, :, :len(vs)] = C.to64(torch.stack(vs)).transpose(1, 0, 2)
        ref = pagedkv.paged_attention(C.to64(q), kc, vc, np.arange(self.B)[:, None], lens,
                                      np.cumsum([0] + counts), self.dim ** -0.5)
        name = {v: n for n, v in C.DT.items()}[self.dt]
        C.check(C.to64(a["out"]), C.to64(a["lse"]), ref, name, self.dim)
        table = self.table.cpu().numpy()
        used = table[table >= 0]
        held = [i for i in self.free[:int(self.count)].tolist()]
        assert len(set(used.tolist())) == len(used)          # no block in two places
        assert not set(used.tolist()) & set(held)            # nor in the pool as well
        assert [(row >= 0).sum() for row in table] == [-(-n // self.bs) for n in lens]

    def roll_back(self, num_drop):
        f, n = self.sv.kv_blocktable_truncate(self.table, self.lens, num_drop, self.bs, 2)
        self.freed, self.num_freed = f, n
        for b, d in enumerate(num_drop.tolist()):
            if d:
                del self.dense[b][0][-d:], self.dense[b][1][-d:]


@pytest.mark.parametrize("bs,dtype", [(16, "bf16"), (4, "f16"), (5, "f32")])
def test_decoding_loop(sv, bs, dtype):
    B, k = 7, 4
    loop = Loop(sv, B, k, bs, dtype, seed=bs, width=-(-80 // bs) + 2)
    g = torch.Generator().manual_seed(99)
    prompts = [11, 1, 30, 17, 16, 5, 24]
    tokens = torch.randint(0, loop.vocab, (sum(prompts),), generator=g).to(DEV)
    loop.step(tokens, prompts)
    dropped = 0
    for step in range(5):
        drafts = torch.randint(0, loop.vocab, (B, k), generator=g).to(DEV, torch.int32)
        last = torch.randint(0, loop.vocab, (B, 1), generator=g).to(DEV, torch.int32)
        window = torch.cat([last, drafts], 1)                 # k + 1 tokens a sequence
        h = loop.step(window.flatten().long(), [k + 1] * B)
        h = h.to(torch.bfloat16).view(B, k + 1, -1)
        noise = torch.randn((B, k, h.shape[2]), generator=g).to(DEV, torch.bfloat16)
        out = sv.spec_verify_lmhead_single((h[:, :k] + 0.05 * noise).contiguous(),
                                           h.contiguous(), loop.head, drafts,
                                           torch.full((B,), 5.0, device=DEV), seed=3, offset=step)
        drop = out["num_drop"]
        assert ((drop >= 0) & (drop <= k)).all()
        loop.roll_back(drop)
        dropped += int(drop.sum())
    assert dropped > 0


def test_loop_in_a_captured_graph(sv):
    """Extend, append and attend captured once and replayed: the state advances by
    itself on the device, replay after replay, as eager calls on a copy do."""
    B, n, bs, heads, kv, dim = 6, 3, 16, 4, 2, 128
    T, width, blocks = B * n + 2, 8, 60
    g = torch.Generator().manual_seed(5)

    def state():
        z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
        s = dict(table=torch.full((B, width), -1, dtype=torch.int32, device=DEV), lens=z(B),
                 new=torch.tensor([3, 0, 1, 3, 2, 3], dtype=torch.int32, device=DEV),
                 free=torch.arange(blocks, dtype=torch.int32, device=DEV),
                 count=torch.tensor([blocks], dtype=torch.int32, device=DEV),
                 kc=z(blocks, kv, bs, dim, dt=torch.bfloat16),
                 vc=z(blocks, kv, bs, dim, dt=torch.bfloat16), qkv=z(T, (heads + 2 * kv) * dim,
                                                                    dt=torch.bfloat16))
        s["e"] = dict(new_lens=s["lens"], num_taken=z(B), free_left=s["count"], cu_tokens=z(B + 1),
                      slot_map=z(T, dt=torch.int64), positions=z(T))
        s["a"] = dict(out=z(T, heads, dim, dt=torch.bfloat16), lse=z(T, heads, dt=torch.float32),
                      workspace=None)
        return s

    def run(s):
        r = sv.kv_blocktable_extend(s["table"], s["lens"], s["new"], s["free"], s["count"], bs, T,
                                    out=s["e"])
        x = s["qkv"]
        k = x[:, heads * dim:(heads + kv) * dim].view(T, kv, dim)
        v = x[:, (heads + kv) * dim:].view(T, kv, dim)
        sv.kv_cache_append(k, v, r["slot_map"], s["kc"], s["vc"])
        sv.kv_paged_attention(x[:, :heads * dim].view(T, heads, dim), s["kc"], s["vc"], s["table"],
                              s["lens"], r["cu_tokens"], out=s["a"])
    a, b = state(), state()
    warm = state()
    run(warm)
    a["a"]["workspace"] = warm["a"]["workspace"]      # both graphs and eager calls may share it
    b["a"]["workspace"] = warm["a"]["workspace"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            run(a)
    for rep in range(12):
        x = torch.randn(a["qkv"].shape, generator=g).to(torch.bfloat16).to(DEV)
        a["qkv"].copy_(x)
        b["qkv"].copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        run(b)
        torch.cuda.synchronize()
        for key in ("table", "lens", "count", "kc", "vc"):
            assert torch.equal(a[key], b[key]), (rep, key)
        rows = int(a["e"]["cu_tokens"][-1])
        assert rows == 12
        assert torch.equal(a["a"]["out"][:rows], b["a"]["out"][:rows])
        assert torch.equal(a["a"]["lse"][:rows], b["a"]["lse"][:rows])
        assert (a["a"]["out"][rows:] == 0).all()               # rows of no sequence
    assert int(a["lens"].max()) == 36


def test_calls_on_two_streams_at_once(sv):
    """Two attention calls in flight with their own workspaces do not disturb each
    other."""
    cases = [C.on_gpu(C.attend_case([6000, 30], [5, 9], 8, 2, 128, 16, "bf16", seed=s))
             for s in (1, 2)]
    names = ("q", "k_cache", "v_cache", "block_table", "seq_lens", "cu_tokens")
    alone = [sv.kv_paged_attention(*[c[n] for n in names])["out"].clone() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(sv.kv_paged_attention(*[cases[i][n] for n in names])["out"])
    torch.cuda.synchronize()
    for i in (0, 1):
        for o in outs[i]:
            assert torch.equal(o, alone[i])


def test_failed_calls_write_nothing(sv):
    """A refusal launches nothing: outputs keep their values."""
    c = C.on_gpu(C.attend_case([30], [4], 4, 2, 64, 16, "bf16"))
    out = torch.full((4, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(sv.SpecVerifyError):
        sv.kv_paged_attention(c["q"], c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"],
                              c["cu_tokens"], scale=-1.0, out=dict(out=out, lse=None, workspace=None))
    lib, kvm = sv.library(), __import__("lossless_token_verification_amd.kv", fromlist=["kv"])
    d = kvm.AppendDesc(3, 2, 64, 0, 4, 1, 0, 0, 0)       # a page of no slots
    p = out.data_ptr()
    assert lib.kv_cache_append(ctypes.byref(d), p, p, p, p, p, None) == sv.SV_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (out == 3.0).all()
