"""The paged cache before a verification: growing block tables, the cache
append, attention over the pages.

Test infrastructure only (see ``oracle/__init__``).

Reading: the counterpart of ``blocktable.kv_blocktable_truncate``.  A sequence
of L tokens that gets n more needs ceil((L + n) / bs) - ceil(L / bs) blocks from
a pool, a stack popped from its end; blocks a rollback freed are pushed first.
Everything below goes one sequence and one token at a time.
"""

import numpy as np

from .blocktable import ceil_div


def blocktable_extend(block_table, seq_lens, num_new, free_blocks, free_count, block_size,
                      max_tokens, freed_blocks=None, num_freed=None):
    """Returns a dict of block_table, free_blocks (the whole array), new_lens,
    num_taken, free_left, cu_tokens, slot_map and positions after the call."""
    table = np.array(block_table, dtype=np.int64, copy=True)
    free = np.array(free_blocks, dtype=np.int64, copy=True)
    B, width = table.shape
    top = min(max(int(free_count), 0), len(free))
    if freed_blocks is not None:
        for b in range(B):
            for i in range(min(max(int(num_freed[b]), 0), np.shape(freed_blocks)[1])):
                if top < len(free):
                    free[top] = freed_blocks[b][i]
                    top += 1
    new_lens, taken, cu = [], [], [0]
    slots = np.full(max_tokens, -1, dtype=np.int64)
    positions = np.full(max_tokens, -1, dtype=np.int64)
    rows, short = 0, False
    for b in range(B):
        L, n = int(seq_lens[b]), int(num_new[b])
        start = rows
        rows += max(n, 0)
        cu.append(min(rows, max_tokens))
        new_lens.append(L)
        if n < 0 or L < 0 or L + n > min(width * block_size, 2 ** 31 - 1) or rows > max_tokens:
            taken.append(-1)
            continue
        first = ceil_div(L, block_size)
        need = ceil_div(L + n, block_size) - first
        if need > 0 and (short or need > top):
            short = True
            taken.append(-2)
            continue
        for i in range(need):
            top -= 1
            table[b, first + i] = free[top]
        taken.append(need)
        new_lens[-1] = L + n
        for j in range(n):
            p = L + j
            slots[start + j] = table[b, p // block_size] * block_size + p % block_size
            positions[start + j] = p
    return dict(block_table=table, free_blocks=free, new_lens=np.array(new_lens, dtype=np.int64),
                num_taken=np.array(taken, dtype=np.int64), free_left=top, cu_tokens=np.array(cu),
                slot_map=slots, positions=positions)


def cache_append(rows, slot_map, cache):
    """The cache [blocks, kv_heads, bs, dim] with each row [T, kv_heads, dim] at its slot."""
    out = np.array(cache, copy=True)
    nb, _, bs, _ = out.shape
    for t, s in enumerate(slot_map):
        if 0 <= s < nb * bs:
            out[s // bs, :, s % bs] = rows[t]
    return out


def paged_attention(q, k_cache, v_cache, block_table, seq_lens, cu_tokens, scale, window=0):
    """float64 attention of each sequence's last tokens.  Returns a dict of out
    [T, H, D] and lse [T, H] (NaN rows: rows of no sequence), and for error bounds
    weight_abs [T, H, D] = sum_t w_t |v_t|, v_max [T, H] the largest |v| seen,
    score_abs [T, H] the largest scale * sum_d |q_d k_d| among the seen keys,
    score_top [T, H] the largest score and keys [T, H] their number."""
    q = np.asarray(q, dtype=np.float64)
    T, H, D = q.shape
    nb, kv, bs, _ = k_cache.shape
    group = H // kv
    nan = np.nan
    r = dict(out=np.full((T, H, D), nan), lse=np.full((T, H), nan),
             weight_abs=np.zeros((T, H, D)), v_max=np.zeros((T, H)), score_abs=np.zeros((T, H)),
             score_top=np.zeros((T, H)), keys=np.zeros((T, H)))
    for b in range(len(seq_lens)):
        t0, t1, L = int(cu_tokens[b]), int(cu_tokens[b + 1]), int(seq_lens[b])
        for t in range(t0, t1):
            p = L - (t1 - t0) + (t - t0)
            end = min(p + 1, block_table.shape[1] * bs)
            seen = [s for s in range(max(0, p - window + 1) if window else 0, end)
                    if 0 <= block_table[b, s // bs] < nb]
            if not seen:
                r["out"][t], r["lse"][t] = 0.0, -np.inf
                continue
            s = np.array(seen)
            page = block_table[b, s // bs]
            for h in range(H):
                k = np.asarray(k_cache[page, h // group, s % bs], dtype=np.float64)
                v = np.asarray(v_cache[page, h // group, s % bs], dtype=np.float64)
                x = scale * (k @ q[t, h])
                m = x.max()
                w = np.exp(x - m)
                z = w.sum()
                r["out"][t, h] = w @ v / z
                r["lse"][t, h] = m + np.log(z)
                r["weight_abs"][t, h] = w @ np.abs(v) / z
                r["v_max"][t, h] = np.abs(v).max()
                r["score_abs"][t, h] = scale * (np.abs(k) @ np.abs(q[t, h])).max()
                r["score_top"][t, h] = m
                r["keys"][t, h] = len(s)
    return r
