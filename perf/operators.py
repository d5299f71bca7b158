"""Timed cases of the paged-KV operators: growing block tables (extend), writing
new keys and values into the pages (append) and the attention of new tokens
over the pages (attend).

A case is a dict of plain values; lengths follow from the case alone, values,
block orders and free lists from the seed.  ``own`` picks the side ``run``
takes: elementary torch operations in 32 bits (False) or the package's calls.
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one request decoding alone: its table grows by a token
        dict(name="extend_token_b1", op="extend", batch=1, ctx_lo=1000, ctx_hi=1000, new_lo=1,
             new_hi=1, block=16, freed=0),
        # a verification step of 256 sequences: 8 drafts and the token before them
        # each, the blocks that the last rollback freed going back to the pool first
        dict(name="extend_verify_b256", op="extend", batch=256, ctx_lo=512, ctx_hi=4096, new_lo=9,
             new_hi=9, block=16, freed=1),
        # 64 prompts admitted at once
        dict(name="extend_prompts_b64", op="extend", batch=64, ctx_lo=0, ctx_hi=0, new_lo=1,
             new_hi=4096, block=16, freed=0),
        # the verification step's keys and values, rows of a fused QKV product
        dict(name="append_verify_b256", op="append", batch=256, ctx_lo=512, ctx_hi=4096, new_lo=9,
             new_hi=9, block=16, heads=32, kv_heads=8, dim=128, dtype="bf16", pad=0),
        # four long prompts
        dict(name="append_prompt_b4", op="append", batch=4, ctx_lo=0, ctx_hi=0, new_lo=4000,
             new_hi=4096, block=16, heads=32, kv_heads=8, dim=128, dtype="bf16", pad=0),
        # odd head count, head size and page size, a batch padded to a fixed row count
        dict(name="append_odd_b37", op="append", batch=37, ctx_lo=0, ctx_hi=777, new_lo=0,
             new_hi=33, block=24, heads=15, kv_heads=5, dim=80, dtype="f16", pad=100),
        # one request decoding alone
        dict(name="attend_token_b1", op="attend", batch=1, ctx_lo=1000, ctx_hi=1000, new_lo=1,
             new_hi=1, block=16, heads=32, kv_heads=8, dim=128, dtype="bf16", window=0, lse=False),
        # the verification step over its contexts
        dict(name="attend_verify_b256", op="attend", batch=256, ctx_lo=512, ctx_hi=4096, new_lo=9,
             new_hi=9, block=16, heads=32, kv_heads=8, dim=128, dtype="bf16", window=0, lse=False),
        # a few requests deep into long contexts, one token each
        dict(name="attend_token_long_b4", op="attend", batch=4, ctx_lo=90000, ctx_hi=131071,
             new_lo=1, new_hi=1, block=16, heads=32, kv_heads=8, dim=128, dtype="bf16", window=0,
             lse=True),
        # chunked prefill on a long context, small heads, float16
        dict(name="attend_chunk_b2", op="attend", batch=2, ctx_lo=15000, ctx_hi=16384, new_lo=500,
             new_hi=512, block=32, heads=16, kv_heads=2, dim=64, dtype="f16", window=0, lse=True),
        # whole prompts, nothing cached before
        dict(name="attend_prompt_b4", op="attend", batch=4, ctx_lo=0, ctx_hi=0, new_lo=2048,
             new_hi=4096, block=16, heads=32, kv_heads=8, dim=128, dtype="bf16", window=0,
             lse=False),
        # prompts and single tokens in one batch, a sliding window, wide heads, odd pages
        dict(name="attend_mixed_b48", op="attend", batch=48, ctx_lo=0, ctx_hi=2000, new_lo=1,
             new_hi=200, block=24, heads=8, kv_heads=8, dim=256, dtype="f16", window=257,
             lse=True),
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """A case that costs no more than the largest listed ones."""
    while True:
        case = _draw(rng)
        cost = work(case)
        if cost["bytes"] < 2.6e9 and cost["flops"] < 3.3e11:
            return case


def _draw(rng):
    op = rng.choice(["extend", "append", "attend", "attend"])
    block = rng.choice([8, 16, 16, 24, 32, 64, 5])
    kind = rng.choice(["tokens", "verify", "prompts"])
    if op == "attend" and kind != "prompts":
        # decoding and verification: any batch, contexts up to the long ones
        batch = _log(rng, 1, 256)
        hi = _log(rng, 17, min(131072, 1000000 // batch))
        new = 1 if kind == "tokens" else rng.randint(2, 16)
        lo, new_lo, new_hi = rng.randint(0, hi), 1 if rng.random() < 0.5 else new, new
    elif op == "attend":
        batch = _log(rng, 1, 16)
        new_hi = _log(rng, 17, 8192 // batch)
        hi = _log(rng, 1, 4096)
        lo, new_lo = rng.randint(0, hi), rng.randint(1, new_hi)
    elif kind == "prompts":
        batch = _log(rng, 1, 64)
        new_hi = _log(rng, 17, 4096 if op == "extend" else 16384 // batch)
        lo, hi, new_lo = 0, rng.randint(0, 100), rng.randint(0, new_hi)
    else:
        batch = _log(rng, 1, 256)
        hi = _log(rng, 17, 4096)
        new_hi = 1 if kind == "tokens" else rng.randint(2, 16)
        lo, new_lo = rng.randint(0, hi), rng.randint(0, new_hi)
    case = dict(op=op, batch=batch, ctx_lo=lo, ctx_hi=hi, new_lo=new_lo, new_hi=new_hi, block=block)
    if op == "extend":
        case["freed"] = rng.randint(0, 1)
        return case
    kv = rng.choice([1, 2, 3, 4, 5, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    case.update(heads=kv * group, kv_heads=kv, dtype=rng.choice(["bf16", "f16"]))
    if op == "append":
        case.update(dim=rng.choice([40, 64, 80, 96, 128, 256]), pad=rng.choice([0, 13]))
        return case
    case.update(dim=rng.choice([64, 128, 128, 256]), lse=rng.random() < 0.5,
                window=rng.choice([0, 0, rng.randint(1, 2000)]))
    return case


def _lengths(case):
    """The contexts and new tokens of a case's sequences."""
    rng = random.Random("%(batch)d %(ctx_lo)d %(ctx_hi)d %(new_lo)d %(new_hi)d" % case)
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    new[0] = max(new[0], 1)
    return ctx, new


def _ceil(a, b):
    return -(-a // b)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _cumulated(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cu


def _tables(lens, block, width, g):
    """Block tables for these lengths, ids in random order; (table, blocks used)."""
    need = [_ceil(n, block) for n in lens]
    total = sum(need)
    order = torch.randperm(max(total, 1), generator=g, device=DEV).to(torch.int32)
    first = _ints(_cumulated(need)[:-1], torch.int64)
    at = torch.arange(width, device=DEV)
    has = at[None] < _ints(need)[:, None]
    table = torch.where(has, order[(first[:, None] + at).clamp(max=max(total - 1, 0))], -1)
    return table.to(torch.int32).contiguous(), total


def _slots(table, ctx, new, block):
    """Slots of the new tokens, packed."""
    seq = _ints([b for b, n in enumerate(new) for _ in range(n)], torch.int64)
    pos = _ints([c + j for c, n in zip(ctx, new) for j in range(n)], torch.int64)
    return table[seq, pos // block].to(torch.int64) * block + pos % block


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    ctx, new = _lengths(case)
    block = case["block"]
    lens = [c + n for c, n in zip(ctx, new)]
    s = dict(op=case["op"], block=block, tokens=sum(new), max_new=max(new), max_len=max(lens))
    if case["op"] == "extend":
        # tables as wide as a request may become, a pool with blocks to spare, and,
        # in a verification loop, the block that each second sequence gave back
        width = _ceil(max(lens), block) + 2
        table, used = _tables(ctx, block, width, g)
        need = sum(_ceil(n, block) - _ceil(c, block) for n, c in zip(lens, ctx))
        freed = case["freed"] * (case["batch"] // 2)
        spare = need + 100
        ids = (torch.randperm(spare + freed, generator=g, device=DEV) + used).to(torch.int32)
        free_blocks = torch.full((spare + freed + 50,), -1, dtype=torch.int32, device=DEV)
        free_blocks[:spare] = ids[:spare]
        s.update(table=table, seq_lens=_ints(ctx), num_new=_ints(new), free_blocks=free_blocks,
                 free_count=_ints([spare]), freed_blocks=None, num_freed=None)
        if case["freed"]:
            back = torch.full((case["batch"], 1), -1, dtype=torch.int32, device=DEV)
            back[1::2, 0] = ids[spare:]
            s.update(freed_blocks=back, num_freed=(back[:, 0] >= 0).to(torch.int32))
        return s
    heads, kv, dim, dt = case["heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    table, used = _tables(lens, block, _ceil(max(lens), block) + 1, g)
    shape = (used + 1, kv, block, dim)
    s.update(k_cache=torch.randn(shape, generator=g, device=DEV, dtype=dt),
             v_cache=torch.randn(shape, generator=g, device=DEV, dtype=dt))
    rows = s["tokens"] + case.get("pad", 0)
    # q, k and v are the three parts of each row of one fused product
    qkv = torch.randn((rows, (heads + 2 * kv) * dim), generator=g, device=DEV, dtype=dt)
    if case["op"] == "append":
        slots = torch.full((rows,), -1, dtype=torch.int64, device=DEV)
        slots[:s["tokens"]] = _slots(table, ctx, new, block)
        s.update(slot_map=slots, k=qkv[:, heads * dim:(heads + kv) * dim].view(rows, kv, dim),
                 v=qkv[:, (heads + kv) * dim:].view(rows, kv, dim))
        return s
    s.update(q=qkv[:, :heads * dim].view(rows, heads, dim), table=table, seq_lens=_ints(lens),
             cu_tokens=_ints(_cumulated(new)), window=case["window"], lse=case["lse"])
    return s


def _plain_extend(s):
    table, lens, n = s["table"], s["seq_lens"].long(), s["num_new"].long()
    block, T, width, free = s["block"], s["tokens"], s["table"].shape[1], s["free_blocks"]
    cum = torch.cumsum(n.clamp(min=0), 0)
    good = (n >= 0) & (lens >= 0) & (lens + n <= width * block) & (cum <= T)
    need = torch.where(good, (lens + n + block - 1) // block - (lens + block - 1) // block, 0)
    off = torch.cumsum(need, 0) - need
    count = s["free_count"].long()
    if s["freed_blocks"] is not None:
        back = s["freed_blocks"]
        m = s["num_freed"].long().clamp(0, back.shape[1])
        at = count + (torch.cumsum(m, 0) - m)[:, None] + torch.arange(back.shape[1], device=DEV)
        keep = torch.arange(back.shape[1], device=DEV)[None] < m[:, None]
        free[at[keep]] = back[keep]
        count = count + m.sum()
    served = good & ((need == 0) | (off + need <= count))
    i = torch.arange(width, device=DEV)[None] - ((lens + block - 1) // block)[:, None]
    mine = served[:, None] & (i >= 0) & (i < need[:, None])
    source = (count - 1 - off[:, None] - i).clamp(0, free.shape[0] - 1)
    table.copy_(torch.where(mine, free[source], table))
    taken = torch.where(served, need, torch.where(good, -2, -1))
    cu = torch.cat([torch.zeros_like(cum[:1]), cum.clamp(max=T)])
    t = torch.arange(T, device=DEV)
    seq = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=len(n) - 1)
    pos = lens[seq] + t - cu[seq]
    has = (t < cu[-1]) & served[seq]
    slot = table[seq, (pos // block).clamp(0, width - 1)].long() * block + pos % block
    return dict(block_table=table, free_blocks=free, new_lens=torch.where(served, lens + n, lens).int(),
                num_taken=taken.int(), free_left=(count - taken.clamp(min=0).sum()).int().view(1),
                cu_tokens=cu.int(), slot_map=torch.where(has, slot, -1),
                positions=torch.where(has, pos, -1).int())


def _plain_append(s):
    slots, block = s["slot_map"], s["block"]
    rows = torch.nonzero(slots >= 0)[:, 0]
    at = slots[rows]
    s["k_cache"][at // block, :, at % block] = s["k"][rows]
    s["v_cache"][at // block, :, at % block] = s["v"][rows]
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_attend(s):
    q, table, block = s["q"], s["table"], s["block"]
    lens, cu = s["seq_lens"].long(), s["cu_tokens"].long()
    T, heads, dim = q.shape
    kv = s["k_cache"].shape[1]
    group, B, n_max = heads // kv, len(lens), s["max_new"]
    n = cu[1:] - cu[:-1]
    j = torch.arange(n_max, device=DEV)
    row = (cu[:-1, None] + j).clamp(max=T - 1)
    pos = (lens - n)[:, None] + j                                   # [B, n_max]
    key = torch.arange(s["max_len"], device=DEV)
    page, at = table[:, key // block].long().clamp(min=0), key % block
    held = (key[None] < lens[:, None])[:, :, None, None]
    k = s["k_cache"][page, :, at[None]].float()                     # [B, keys, kv, dim]
    v = torch.where(held, s["v_cache"][page, :, at[None]].float(), 0.0)
    k, v = k.permute(0, 2, 3, 1).contiguous(), v.permute(0, 2, 1, 3).contiguous()
    qp = q[row].float().view(B, n_max, kv, group, dim).permute(0, 2, 1, 3, 4)
    score = torch.matmul(qp.reshape(B, kv, n_max * group, dim), k) * dim ** -0.5
    del k
    score = score.view(B, kv, n_max, group, -1)
    seen = (key <= pos[:, :, None]) & (key < lens[:, None, None])
    if s["window"]:
        seen &= key > pos[:, :, None] - s["window"]
    score.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, kv, n_max * group, -1), v).view(B, kv, n_max, group, dim)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (total.log() + top)[..., 0]
    mine = j[None] < n[:, None]
    out = dict(out=o.permute(0, 2, 1, 3, 4).reshape(B, n_max, heads, dim)[mine].to(q.dtype))
    if s["lse"]:
        out["lse"] = lse.permute(0, 2, 1, 3).reshape(B, n_max, heads)[mine]
    return out


def _own_run(s):
    import lossless_token_verification_amd as sv
    if s["op"] == "extend":
        r = sv.kv_blocktable_extend(s["table"], s["seq_lens"], s["num_new"], s["free_blocks"],
                                    s["free_count"], s["block"], s["tokens"],
                                    freed_blocks=s["freed_blocks"], num_freed=s["num_freed"],
                                    out=s.get("out"))
        s["out"] = r   # a loop reuses its output tensors
        return dict(r, block_table=s["table"], free_blocks=s["free_blocks"])
    if s["op"] == "append":
        sv.kv_cache_append(s["k"], s["v"], s["slot_map"], s["k_cache"], s["v_cache"])
        return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    r = sv.kv_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq_lens"],
                              s["cu_tokens"], sliding_window=s["window"], max_new=s["max_new"],
                              lse=s["lse"])
    return dict(out=r["out"], lse=r["lse"]) if s["lse"] else dict(out=r["out"])


def run(state):
    if own:
        return _own_run(state)
    return {"extend": _plain_extend, "append": _plain_append, "attend": _plain_attend}[state["op"]](state)


def _keys(case):
    """Keys read (once for each sequence) and (row, key) pairs of an attention case."""
    w, keys, pairs = case["window"], 0, 0
    for c, n in zip(*_lengths(case)):
        keys += (c + n) - (max(0, c + 1 - w) if w else 0) if n else 0
        for p in range(c, c + n):
            pairs += min(p + 1, w) if w else p + 1
    return keys, pairs


def work(case):
    ctx, new = _lengths(case)
    T, B, block = sum(new), case["batch"], case["block"]
    if case["op"] == "extend":
        need = sum(_ceil(c + n, block) - _ceil(c, block) for c, n in zip(ctx, new))
        # lengths in and out, counts, offsets; block ids popped and written; 12 bytes a token
        return dict(bytes=B * 20 + need * 8 + T * 12 + case["freed"] * (B // 2) * 8, flops=0)
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "append":
        return dict(bytes=T * (case["kv_heads"] * case["dim"] * size * 4 + 8), flops=0)
    keys, pairs = _keys(case)
    moved = keys * case["kv_heads"] * case["dim"] * size * 2 + T * case["heads"] * case["dim"] * size * 2
    return dict(bytes=moved + _ceil(keys, block) * 4 + B * 8 + (T * case["heads"] * 4 if case["lse"] else 0),
                flops=4 * case["dim"] * case["heads"] * pairs)


def _placed(cache, rows, slots):
    """The cache in 64 bits with each row at its slot, seen as one list of slots."""
    pages, kv, block, dim = cache.shape
    flat = cache.double().transpose(1, 2).reshape(pages * block, kv, dim)
    flat = torch.cat([flat, flat[:1]])           # a place of its own for rows without one
    flat[torch.where(slots < 0, pages * block, slots)] = rows.double()
    return flat[:-1].view(pages, block, kv, dim).transpose(1, 2)


def exact(case, seed):
    """Attention by its definition in 64 bits, a sequence and a key head at a time;
    the rows that an append puts in place; a block table has no computed numbers."""
    if case["op"] == "extend":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return {name: _placed(s[name], s[name[0]], s["slot_map"]) for name in ("k_cache", "v_cache")}
    ctx, new = _lengths(case)
    T, heads, dim = s["q"].shape
    kv = case["kv_heads"]
    per = heads // kv
    out = torch.zeros((T, heads, dim), dtype=torch.float64, device=DEV)
    lse = torch.full((T, heads), -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b in range(case["batch"]):
        L = ctx[b] + new[b]
        pages = s["table"][b, :_ceil(L, case["block"])].long()
        where = torch.arange(L, device=DEV)
        for h in range(kv):
            k = s["k_cache"][pages, h].reshape(-1, dim)[:L].double()
            v = s["v_cache"][pages, h].reshape(-1, dim)[:L].double()
            for r0 in range(0, new[b], 2048):
                r1 = min(new[b], r0 + 2048)
                p = torch.arange(ctx[b] + r0, ctx[b] + r1, device=DEV)[:, None]
                hidden = where > p
                if case["window"]:
                    hidden |= where <= p - case["window"]
                for e in range(h * per, (h + 1) * per):
                    x = s["q"][at + r0:at + r1, e].double() @ k.T / math.sqrt(dim)
                    x[hidden] = -math.inf
                    z = torch.logsumexp(x, 1)
                    out[at + r0:at + r1, e] = torch.exp(x - z[:, None]) @ v
                    lse[at + r0:at + r1, e] = z
        at += new[b]
    return dict(out=out, lse=lse) if case["lse"] else dict(out=out)
