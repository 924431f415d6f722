"""Plain float64 forms of the paged-cache step: plan, append, attention over a prefix and own pages.

TEST INFRASTRUCTURE ONLY, like the rest of this package: written from the definitions, one
request, one token and one row at a time, sharing no code with the product path.
"""
from __future__ import annotations

import numpy as np

PAGE = 128


def page_plan(ctx_lens, new_lens, free_pages, free_head, block_table, max_tokens):
    """(block_table, seq_lens, cu_new, slot_map, free_head): every new token takes the next row of its
    request's last page, or the first row of the next free page."""
    table = np.array(block_table, dtype=np.int32)
    head, cu, slots = int(free_head), [0], []
    for b, (c, n) in enumerate(zip(ctx_lens, new_lens)):
        for pos in range(int(c), int(c) + int(n)):
            if pos % PAGE == 0:
                table[b, pos // PAGE] = free_pages[head]
                head += 1
            slots.append(int(table[b, pos // PAGE]) * PAGE + pos % PAGE)
        cu.append(cu[-1] + int(n))
    slots += [-1] * (max_tokens - len(slots))
    seq = np.asarray(ctx_lens, dtype=np.int32) + np.asarray(new_lens, dtype=np.int32)
    return table, seq, np.array(cu, dtype=np.int32), np.array(slots, dtype=np.int32), head


def kv_append(new, slots, pages):
    """Copies row t of ``new`` (N, Hkv, d) to row slots[t] % 128 of page slots[t] // 128; negative slots are skipped."""
    out = np.array(pages)
    for t, s in enumerate(slots):
        if s >= 0:
            out[s // PAGE, :, s % PAGE] = new[t]
    return out


def gather(pages, table, length):
    """(length, Hkv, d): the rows of a sequence whose page i is table[i]."""
    return np.array([pages[table[j // PAGE], :, j % PAGE] for j in range(length)]).reshape(length, *np.shape(pages)[1::2])


def row(q, k, v, scale):
    """One row over its visible keys: (o, lse, spread, size).

    spread_c = sqrt(sum_j w_j (v_jc - o_c)^2), at least sum_j w_j |v_jc - o_c| (the weights sum to 1);
    size = the largest scale * sum_c |q_c k_jc| (bounds the rounding of a score).
    """
    d = q.shape[0]
    if k.shape[0] == 0:
        return np.zeros(d), -np.inf, np.zeros(d), 0.0
    s = scale * (k @ q)
    m = s.max()
    e = np.exp(s - m)
    w = e / e.sum()
    o = w @ v
    return o, m + np.log(e.sum()), np.sqrt(w @ (v - o) ** 2), float((scale * (np.abs(k) @ np.abs(q))).max())


def attention_prefix_paged(q, k_pages, v_pages, prefix_table, prefix_len, block_table, seq_lens, cu_new, causal, scale):
    """(O, LSE, spread, size) of every row (n, h); rows behind the last request come back as NaN."""
    N, H, d = q.shape
    group = H // k_pages.shape[1]
    O, spread = np.full((N, H, d), np.nan), np.zeros((N, H, d))
    lse, size = np.full((N, H), np.nan), np.zeros((N, H))
    kp, vp = (gather(x, prefix_table, prefix_len) for x in (k_pages, v_pages))
    for b, n in enumerate(seq_lens):
        t = int(cu_new[b + 1] - cu_new[b])
        if t == 0:
            continue
        ko, vo = (gather(x, block_table[b], int(n)) for x in (k_pages, v_pages))
        for i in range(t):
            seen = max(0, min(int(n), int(n) - t + i + 1)) if causal else int(n)
            for h in range(H):
                g, r = h // group, int(cu_new[b]) + i
                k, v = (np.concatenate([x[:, g], y[:seen, g]]) for x, y in ((kp, ko), (vp, vo)))
                O[r, h], lse[r, h], spread[r, h], size[r, h] = row(q[r, h], k, v, scale)
    return O, lse, spread, size
