"""Float64 oracle of the paged key-value cache calls (numpy, one request and
one token at a time).  It shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def plan(kv_len, written, accepted_len, release, new_len, table, pages, free, count, page_size,
         max_new):
    """sv_kv_plan for valid inputs: lists in, a dict of new state out."""
    B = len(kv_len)
    table = [list(r) for r in table]
    free = list(free)
    base, need, want = [], [], []
    for b in range(B):
        w = written[b] if written is not None else 0
        if w <= 0:
            stay = 0
        elif accepted_len is None:
            stay = w
        else:
            stay = accepted_len[b] + 1 if accepted_len[b] >= 0 else 0
        gone = release is not None and release[b] != 0
        base.append(0 if gone else kv_len[b] + stay)
        want.append(0 if gone else new_len[b])
        need.append(-(-(base[b] + want[b]) // page_size))
    for b in range(B):
        for j in range(need[b], pages[b]):
            free[count] = table[b][j]
            count += 1
    q_len, held, starved = list(want), list(pages), False
    for b in range(B):
        lack = need[b] - pages[b]
        if lack > 0 and (starved or lack > count):
            starved, q_len[b] = True, 0
            continue
        for j in range(pages[b], need[b]):
            count -= 1
            table[b][j] = free[count]
        held[b] = need[b]
    slots = np.full((B, max_new), -1, np.int64)
    pos = np.full((B, max_new), -1, np.int32)
    for b in range(B):
        for i in range(q_len[b]):
            t = base[b] + i
            pos[b, i] = t
            slots[b, i] = table[b][t // page_size] * page_size + t % page_size
    return dict(kv_len=np.array(base, np.int32), pages=np.array(held, np.int32), free_count=count,
                q_len=np.array(q_len, np.int32), slot_map=slots, positions=pos,
                block_table=np.array(table, np.int32).reshape(B, -1),
                free_pages=np.array(free, np.int32), starved=starved)


def ancestors(parents, i):
    """i and the nodes above it; parents None: a chain."""
    out = []
    while i >= 0:
        out.append(i)
        i = i - 1 if parents is None else int(parents[i])
    return out


def attend(q, k, v, table, kv_len, q_len, parents, scale):
    """q [B, n, hq, d]; k, v [pages, page_size, heads, d]; float64 out, lse,
    and per row the largest |scale| sum |q k| and the sum of p |v|, from which
    rounding errors are bounded."""
    B, n, hq, d = q.shape
    page, heads = k.shape[1], k.shape[2]
    g = hq // heads
    out = np.zeros((B, n, hq, d))
    lse = np.full((B, n, hq), -np.inf)
    size = np.zeros((B, n, hq))
    absv = np.zeros((B, n, hq, d))
    for b in range(B):
        a = int(kv_len[b])
        for i in range(int(q_len[b])):
            seen = list(range(a)) + [a + j for j in
                                     ancestors(None if parents is None else parents[b], i)]
            seen = np.array(sorted(seen))
            pg, off = np.asarray(table[b])[seen // page], seen % page
            for x in range(hq):
                kk = k[pg, off, x // g].astype(np.float64)
                vv = v[pg, off, x // g].astype(np.float64)
                qq = q[b, i, x].astype(np.float64)
                z = scale * (kk @ qq)
                m = z.max()
                w = np.exp(z - m)
                out[b, i, x] = (w @ vv) / w.sum()
                lse[b, i, x] = m + np.log(w.sum())
                size[b, i, x] = abs(scale) * (np.abs(kk) @ np.abs(qq)).max()
                absv[b, i, x] = (w @ np.abs(vv)) / w.sum()
    return out, lse, size, absv


def commit(cache, table, kv_len, nodes, accepted_len):
    """cache [layers, pages, page_size, heads, d]: the cache afterwards."""
    page = cache.shape[2]
    out = cache.copy()
    for b in range(len(kv_len)):
        for i in range(1, int(accepted_len[b]) + 1):
            s, t = int(kv_len[b]) + int(nodes[b][i]), int(kv_len[b]) + i
            out[:, table[b][t // page], t % page] = cache[:, table[b][s // page], s % page]
    return out
