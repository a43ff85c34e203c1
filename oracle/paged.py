"""Float64 reference of the paged key-value cache operators: page plan, RoPE
and append, attention over pages. Plain loops over requests, rows and heads.
"""

import torch

F64 = torch.float64


def page_plan(lens, starts, tables, held, free, n_free, page, n_rows):
    """Lists in, a dict of lists out: releases in request and table order onto
    the stack, then grants in request order until one does not fit."""
    B, W = len(lens), len(tables[0])
    tables, free, held = [list(t) for t in tables], list(free), list(held)
    free_top = n_free
    need, status = [0] * B, [0] * B
    for b in range(B):
        need[b] = -(-lens[b] // page)
        if lens[b] < 0 or need[b] > W or starts[b + 1] - starts[b] > lens[b] or not 0 <= held[b] <= W:
            status[b], need[b] = 2, held[b]
        for i in range(need[b], held[b]):
            free[free_top] = tables[b][i]
            free_top += 1
    served = True
    for b in range(B):
        want = need[b] - held[b]
        if want > 0:
            served = served and want <= free_top
            if not served:
                status[b], need[b] = 1, held[b]
                continue
            for i in range(held[b], need[b]):
                free_top -= 1
                tables[b][i] = free[free_top]
        held[b] = need[b]
    slots, positions = [-1] * n_rows, [0] * n_rows
    for b in range(B):
        if status[b] == 0:
            for i in range(max(0, starts[b]), min(n_rows, starts[b + 1])):
                p = lens[b] - (starts[b + 1] - i)
                positions[i], slots[i] = p, tables[b][p // page] * page + p % page
    return dict(tables=tables, held=held, free=free, n_free=free_top, status=status, slots=slots, positions=positions)


def rotate(x, cs):
    """Rotate-half RoPE of one head vector x [hd] by cs [hd / 2][2]."""
    x, cs = x.to(F64), cs.to(F64)
    h = x.shape[0] // 2
    return torch.cat([x[:h] * cs[:, 0] - x[h:] * cs[:, 1], x[h:] * cs[:, 0] + x[:h] * cs[:, 1]])


def attention(q, k, v, scale, seen):
    """One query row of one head: q [hd], k and v [n, hd], seen bool [n].
    Returns (out, lse, sum of p |v|, largest sum of |q k| * scale)."""
    q, k, v = q.to(F64), k[seen].to(F64), v[seen].to(F64)
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[0], dtype=F64)
        return z, float("-inf"), z, 0.0
    x = (k @ q) * scale
    lse = torch.logsumexp(x, 0)
    p = torch.exp(x - lse)
    return p @ v, float(lse), p @ v.abs(), float(((k.abs() @ q.abs()) * abs(scale)).max())


def gather(cache, table, n, page, head):
    """Slots 0 .. n - 1 of a request, [n, hd], from cache [pages, heads, page,
    hd]; a table entry outside the cache reads as zeros."""
    rows = []
    for s in range(n):
        pg = int(table[s // page])
        rows.append(cache[pg, head, s % page] if 0 <= pg < cache.shape[0] else torch.zeros_like(cache[0, 0, 0]))
    return torch.stack(rows) if rows else cache.new_zeros((0, cache.shape[3]))


def paged_attention(q, k_cache, v_cache, tables, lens, starts, scale, mask=None, max_rows=80):
    """All rows: (out [n, heads, hd], lse [n, heads], a [n, heads, hd],
    qk [n, heads], live [n]); rows outside every request are not live."""
    n, nq, hd = q.shape
    nkv, page = k_cache.shape[1], k_cache.shape[2]
    W = len(tables[0])
    out, a = torch.zeros(n, nq, hd, dtype=F64), torch.zeros(n, nq, hd, dtype=F64)
    lse, qk = torch.full((n, nq), float("-inf"), dtype=F64), torch.zeros(n, nq, dtype=F64)
    live = torch.zeros(n, dtype=torch.bool)
    for b, ln in enumerate(lens):
        ln = max(0, min(ln, W * page))
        rows = starts[b + 1] - starts[b]
        first = ln - rows
        for kvh in range(nkv):
            k = gather(k_cache, tables[b], ln, page, kvh)
            v = gather(v_cache, tables[b], ln, page, kvh)
            for j in range(min(rows, max_rows)):
                i = starts[b] + j
                live[i] = True
                seen = torch.zeros(ln, dtype=torch.bool)
                seen[:max(0, first)] = True
                for c in range(rows):
                    if first + c >= 0 and c < 64 if mask is not None else first + c >= 0:
                        seen[first + c] = c <= j if mask is None else bool((int(mask[i]) >> c) & 1)
                for h in range(kvh * (nq // nkv), (kvh + 1) * (nq // nkv)):
                    out[i, h], lse[i, h], a[i, h], qk[i, h] = attention(q[i, h], k, v, scale, seen)
    return out, lse, a, qk, live
