"""The rotated append and the 4-bit cache as a decoding loop uses them, around the
LM-head verification: extend the tables for the drafted window, turn and write its
rows, attend, verify, roll back what was rejected, take the freed blocks back.  The toy
model and its state are test_gpu_kv_loop's; every step is checked against dense
copies made by the oracle."""

import numpy as np
import pytest
import torch

from oracle import kvq4, pagedkv
from tests import kvcases as C
from tests import kvq4cases as Q
from tests.test_gpu_kv_loop import DEV, Loop, sv   # noqa: F401
from tests.test_gpu_kv_rotary import table, turned_bound

pytestmark = pytest.mark.gpu


class Turned(Loop):
    """Rotated rows in the 16-bit cache (bits 16) or in the 4-bit one (bits 4)."""

    def __init__(self, bits, *args, **kw):
        super().__init__(*args, **kw)
        self.bits, self.cs = bits, table(400, self.dim).to(DEV)
        if bits == 4:
            self.cache = self.sv.make_kv_cache_q4(self.kc.shape[0], self.kv, self.bs, self.dim, DEV)
            self.cache["k_scales"].fill_(255)
            self.cache["v_scales"].fill_(float("nan"))

    def step(self, tokens, counts):
        sv, T, dim = self.sv, sum(counts), self.dim   # noqa: F811
        new = torch.tensor(counts, dtype=torch.int32, device=DEV)
        r = sv.kv_blocktable_extend(self.table, self.lens, new, self.free, self.count, self.bs, T,
                                    freed_blocks=self.freed, num_freed=self.num_freed)
        self.lens, self.count = r["new_lens"], r["free_left"]
        self.num_freed.zero_()
        x = torch.matmul(self.embed[tokens], self.wqkv)
        H, kvd = self.heads * dim, self.kv * dim
        q, k, v = (x[:, a:a + n].view(T, -1, dim) for a, n in ((0, H), (H, kvd), (H + kvd, kvd)))
        turn = dict(positions=r["positions"], cos_sin=self.cs)
        if self.bits == 4:
            tq = sv.kv_cache_append_q4(k, v, r["slot_map"], self.cache, q=q, **turn)
            a = sv.kv_paged_attention_q4(tq, self.cache, self.table, self.lens, r["cu_tokens"],
                                         lse=True, max_new=max(counts))
            held = sv.kv_cache_read_q4(r["slot_map"], self.cache, torch.float32)
        else:
            tq = sv.kv_cache_append_rotary(q, k, v, r["positions"], self.cs, r["slot_map"], self.kc,
                                           self.vc)
            a = sv.kv_paged_attention(tq, self.kc, self.vc, self.table, self.lens, r["cu_tokens"],
                                      lse=True, max_new=max(counts))
            slot = r["slot_map"]
            held = tuple(c[slot // self.bs, :, slot % self.bs] for c in (self.kc, self.vc))
        torch.cuda.synchronize()
        # the rows: turned by their positions, and as the oracle stores them
        name = {t: n for n, t in C.DT.items()}[self.dt]
        pos, cs = r["positions"].tolist(), self.cs.cpu().numpy().astype(np.float64)
        assert pos == [p for b, n in enumerate(counts)
                       for p in range(len(self.dense[b][0]), len(self.dense[b][0]) + n)]
        ref_q, ref_k = (kvq4.rotate(C.to64(t), pos, cs, False) for t in (q, k))
        assert (np.abs(C.to64(tq) - ref_q) <= turned_bound(C.to64(q), cs, pos, False, name)).all()
        if self.bits == 4:
            rows = Q.quantised(torch.from_numpy(ref_k).float(), v.cpu().float())
            ref_k = kvq4.key_values(rows["k_codes"].numpy(), rows["k_scales"].numpy())
            ref_v = kvq4.value_values(rows["v_codes"].numpy(), rows["v_scales"].numpy())
            assert np.array_equal(C.to64(held[0]), ref_k)
            assert np.array_equal(C.to64(held[1]), ref_v.astype(np.float32))
        else:
            assert (np.abs(C.to64(held[0]) - ref_k) <=
                    turned_bound(C.to64(k), cs, pos, False, name)).all()
            assert torch.equal(held[1], v)
        at = 0
        for b, n in enumerate(counts):
            for i in (0, 1):
                self.dense[b][i] += list(held[i][at:at + n].cpu())
            at += n
        if self.bits == 4:
            case = dict(q=tq.cpu(), cache={n: t.cpu() for n, t in self.cache.items()},
                        block_table=self.table.cpu(), seq_lens=self.lens.cpu(),
                        cu_tokens=r["cu_tokens"].cpu())
            ref = Q.reference(case)
            Q.check(C.to64(a["out"]), C.to64(a["lse"]), ref, name, dim)
            self.agree(tq, ref, counts)
        else:
            self.check(tq, a, counts)
        return a["out"].reshape(T, H)

    def agree(self, q, ref, counts):
        """The pages hold what the dense copies hold."""
        width = max(len(d[0]) for d in self.dense)
        both = np.zeros((2, self.B, self.kv, width, self.dim))
        for b, d in enumerate(self.dense):
            for i in (0, 1):
                both[i, b, :, :len(d[i])] = C.to64(torch.stack(d[i])).transpose(1, 0, 2)
        dense = pagedkv.paged_attention(C.to64(q), both[0], both[1], np.arange(self.B)[:, None],
                                        [len(d[0]) for d in self.dense], np.cumsum([0] + counts),
                                        self.dim ** -0.5)
        assert np.allclose(dense["out"], ref["out"], rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("bits,bs,dtype", [(16, 16, "bf16"), (16, 5, "f32"), (4, 16, "bf16"),
                                           (4, 5, "f16")])
def test_decoding_loop(sv, bits, bs, dtype):   # noqa: F811
    B, k = 7, 4
    loop = Turned(bits, sv, B, k, bs, dtype, seed=bs, width=-(-80 // bs) + 2)
    g = torch.Generator().manual_seed(99)
    prompts = [11, 1, 30, 17, 16, 5, 24]
    loop.step(torch.randint(0, loop.vocab, (sum(prompts),), generator=g).to(DEV), prompts)
    dropped = 0
    for step in range(4):
        drafts = torch.randint(0, loop.vocab, (B, k), generator=g).to(DEV, torch.int32)
        last = torch.randint(0, loop.vocab, (B, 1), generator=g).to(DEV, torch.int32)
        h = loop.step(torch.cat([last, drafts], 1).flatten().long(), [k + 1] * B)
        h = h.to(torch.bfloat16).view(B, k + 1, -1)
        noise = torch.randn((B, k, h.shape[2]), generator=g).to(DEV, torch.bfloat16)
        out = sv.spec_verify_lmhead_single((h[:, :k] + 0.05 * noise).contiguous(),
                                           h.contiguous(), loop.head, drafts,
                                           torch.full((B,), 5.0, device=DEV), seed=3, offset=step)
        assert ((out["num_drop"] >= 0) & (out["num_drop"] <= k)).all()
        loop.roll_back(out["num_drop"])
        dropped += int(out["num_drop"].sum())
    assert dropped > 0


@pytest.mark.parametrize("bits", [16, 4])
def test_loop_in_a_captured_graph(sv, bits):   # noqa: F811
    """Extend, turn, append, attend and roll back captured once and replayed: the state
    advances by itself on the device, replay after replay, as eager calls on a copy do.
    The batch is padded: rows behind the last sequence have no slot."""
    B, bs, heads, kv, dim = 6, 16, 4, 2, 128
    T, width, blocks = B * 3 + 2, 8, 60
    g = torch.Generator().manual_seed(5)
    cs = table(300, dim).to(DEV)
    drop = torch.tensor([1, 0, 1, 0, 2, 0], dtype=torch.int32, device=DEV)

    def state():
        z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
        b16 = torch.bfloat16
        s = dict(table=torch.full((B, width), -1, dtype=torch.int32, device=DEV), lens=z(B),
                 new=torch.tensor([3, 0, 1, 3, 2, 3], dtype=torch.int32, device=DEV),
                 free=torch.arange(blocks, dtype=torch.int32, device=DEV),
                 count=torch.tensor([blocks], dtype=torch.int32, device=DEV),
                 freed=z(B, 2), num_freed=z(B), qkv=z(T, (heads + 2 * kv) * dim, dt=b16),
                 tq=z(T, heads, dim, dt=b16))
        s["cache"] = (sv.make_kv_cache_q4(blocks, kv, bs, dim, DEV) if bits == 4 else
                      dict(kc=z(blocks, kv, bs, dim, dt=b16), vc=z(blocks, kv, bs, dim, dt=b16)))
        s["e"] = dict(new_lens=s["lens"], num_taken=z(B), free_left=s["count"], cu_tokens=z(B + 1),
                      slot_map=z(T, dt=torch.int64), positions=z(T))
        s["a"] = dict(out=z(T, heads, dim, dt=b16), lse=z(T, heads, dt=torch.float32), workspace=None)
        return s

    def run(s):
        r = sv.kv_blocktable_extend(s["table"], s["lens"], s["new"], s["free"], s["count"], bs, T,
                                    freed_blocks=s["freed"], num_freed=s["num_freed"], out=s["e"])
        q, k, v = (s["qkv"][:, a * dim:(a + n) * dim].view(T, n, dim)
                   for a, n in ((0, heads), (heads, kv), (heads + kv, kv)))
        if bits == 4:
            sv.kv_cache_append_q4(k, v, r["slot_map"], s["cache"], q=q, positions=r["positions"],
                                  cos_sin=cs, out=s["tq"])
            sv.kv_paged_attention_q4(s["tq"], s["cache"], s["table"], s["lens"], r["cu_tokens"],
                                     out=s["a"])
        else:
            sv.kv_cache_append_rotary(q, k, v, r["positions"], cs, r["slot_map"], s["cache"]["kc"],
                                      s["cache"]["vc"], out=s["tq"])
            sv.kv_paged_attention(s["tq"], s["cache"]["kc"], s["cache"]["vc"], s["table"], s["lens"],
                                  r["cu_tokens"], out=s["a"])
        f, n = sv.kv_blocktable_truncate(s["table"], s["lens"], drop, bs, 2)
        s["freed"].copy_(f)
        s["num_freed"].copy_(n)
    a, b, warm = state(), state(), state()
    run(warm)
    a["a"]["workspace"] = b["a"]["workspace"] = warm["a"]["workspace"]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            run(a)
    for rep in range(10):
        x = torch.randn(a["qkv"].shape, generator=g).to(torch.bfloat16).to(DEV)
        for s in (a, b):
            s["qkv"].copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        run(b)
        torch.cuda.synchronize()
        for key in ("table", "lens", "count", "tq"):
            assert torch.equal(a[key], b[key]), (rep, key)
        for n in a["cache"]:
            assert torch.equal(a["cache"][n], b["cache"][n]), (rep, n)
        rows = int(a["e"]["cu_tokens"][-1])
        assert rows == 12
        assert torch.equal(a["a"]["out"][:rows], b["a"]["out"][:rows])
        assert torch.equal(a["a"]["lse"][:rows], b["a"]["lse"][:rows])
        assert (a["a"]["out"][rows:] == 0).all()               # rows of no sequence
    assert a["lens"].tolist() == [20, 0, 0, 30, 0, 30]


def test_appends_on_two_streams_at_once(sv):   # noqa: F811
    """Two appends in flight into parts of one cache that do not meet."""
    T, kv, heads, dim, bs, blocks = 700, 2, 8, 128, 16, 100
    g = torch.Generator().manual_seed(8)
    cs = table(300, dim).to(DEV)
    rows = [torch.randn((T, heads + 2 * kv, dim), generator=g).bfloat16().to(DEV) for _ in (0, 1)]
    slots = [(torch.randperm(800, generator=g)[:T] + 800 * i).to(DEV) for i in (0, 1)]
    pos = torch.randint(0, 300, (T,), generator=g, dtype=torch.int32).to(DEV)

    def append(i, cache):
        q, k, v = (rows[i][:, a:a + n] for a, n in ((0, heads), (heads, kv), (heads + kv, kv)))
        return sv.kv_cache_append_q4(k, v, slots[i], cache, q=q, positions=pos, cos_sin=cs)
    one = sv.make_kv_cache_q4(blocks, kv, bs, dim, DEV)
    alone = [append(i, one).clone() for i in (0, 1)]
    both = sv.make_kv_cache_q4(blocks, kv, bs, dim, DEV)
    streams = [torch.cuda.Stream() for _ in (0, 1)]
    torch.cuda.synchronize()
    for _ in range(10):
        outs = []
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs.append(append(i, both))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))
        assert all(torch.equal(one[n], both[n]) for n in one)
        for t in both.values():
            t.zero_()
        torch.cuda.synchronize()
