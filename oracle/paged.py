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


def chunk_attention(q, k_cache, v_cache, tables, lens, starts, scale):
    """As paged_attention without a mask, a KV head's rows of a request at a
    time: (out, lse, a, qk, live)."""
    n, nq, hd = q.shape
    nkv, page = k_cache.shape[1], k_cache.shape[2]
    g = nq // nkv
    out, a = torch.zeros(n, nq, hd, dtype=F64), torch.zeros(n, nq, hd, dtype=F64)
    lse, qk = torch.full((n, nq), float("-inf"), dtype=F64), torch.zeros(n, nq, dtype=F64)
    live = torch.zeros(n, dtype=torch.bool)
    for b, ln in enumerate(lens):
        ln = max(0, min(ln, len(tables[0]) * page))
        s, e = starts[b], starts[b + 1]
        live[s:e] = True
        first = ln - (e - s)                                   # position of row s
        at = max(s, s - first)                                 # rows in front of it see nothing
        if at >= e:
            continue
        pos = torch.arange(first + at - s, ln)
        unseen = torch.arange(ln)[None] > pos[:, None]
        for h in range(nkv):
            k, v = (gather(c, tables[b], ln, page, h).to(F64) for c in (k_cache, v_cache))
            x = q[at:e, h * g:(h + 1) * g].to(F64).transpose(0, 1) @ k.t() * scale          # [g, rows, ln]
            m = q[at:e, h * g:(h + 1) * g].to(F64).abs().transpose(0, 1) @ k.abs().t() * abs(scale)
            x = x.masked_fill(unseen, float("-inf"))
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - z[..., None])
            out[at:e, h * g:(h + 1) * g] = (p @ v).transpose(0, 1)
            a[at:e, h * g:(h + 1) * g] = (p @ v.abs()).transpose(0, 1)
            lse[at:e, h * g:(h + 1) * g] = z.t()
            qk[at:e, h * g:(h + 1) * g] = m.masked_fill(unseen, 0.0).amax(-1).t()
    return out, lse, a, qk, live


def page_free(requests, keep, tables, held, shares, free, n_free, page):
    """Lists in, a dict of lists out (tables is not changed)."""
    B, W, P = len(held), len(tables[0]), len(shares)
    held, free = list(held), list(free)
    holders = [s + 1 for s in shares]
    status, released, named = [], [], set()
    for r, k in zip(requests, keep or [0] * len(requests)):
        first = -(-k // page)
        bad = not 0 <= r < B or r in named or k < 0 or not 0 <= held[r] <= W or first > held[r]
        if 0 <= r < B:
            named.add(r)
        if not bad and k % page and 0 <= tables[r][first - 1] < P:
            bad = shares[tables[r][first - 1]] > 0
        status.append(2 if bad else 0)
        if not bad:
            released += [p for p in tables[r][first:held[r]] if 0 <= p < P]
            held[r] = first
    for p in released:
        holders[p] -= 1
    top = n_free
    for i, p in enumerate(released):
        if holders[p] <= 0 and p not in released[:i]:
            free[top] = p
            top += 1
    return dict(held=held, shares=[max(h - 1, 0) for h in holders], free=free, n_free=top, status=status)


def page_fork(src, dst, lens, tables, held, shares, free, n_free, page):
    """Lists in, a dict of lists out."""
    B, W, P = len(held), len(tables[0]), len(shares)
    tables, new_held, shares, top = [list(t) for t in tables], list(held), list(shares), n_free
    res = dict(source=[], target=[], slots=[], status=[])
    named, short = set(), False
    for s, d in zip(src, dst):
        bad = not (0 <= s < B and 0 <= d < B) or s == d or d in named or held[d] != 0
        bad = bad or lens[s] < 0 or held[s] > W or -(-lens[s] // page) > held[s]
        named.add(d)
        part = 0 if bad else lens[s] % page
        short = short or (part > 0 and top == 0)
        status = 2 if bad else 1 if part and short else 0
        source, target = -1, -1
        if status == 0:
            full = lens[s] // page
            for j in range(full):
                tables[d][j] = tables[s][j]
                if 0 <= tables[s][j] < P:
                    shares[tables[s][j]] += 1
            if part:
                top -= 1
                source, target = tables[s][full], free[top]
                tables[d][full] = target
            new_held[d] = -(-lens[s] // page)
        for name, x in (("source", source), ("target", target), ("slots", part if target >= 0 else 0), ("status", status)):
            res[name].append(x)
    return dict(tables=tables, held=new_held, shares=shares, n_free=top, **res)


def page_compact(tables, held, shares):
    """Lists in, a dict of lists out."""
    P = len(shares)
    live = sorted({p for t, h in zip(tables, held) for p in t[:h] if 0 <= p < P})
    u = len(live)
    source, target = [p for p in live if p >= u], [p for p in range(u) if p not in set(live)]
    to = dict(zip(source, target))
    new = [0] * P
    for p in live:
        new[to.get(p, p)] = shares[p]
    return dict(tables=[[to.get(p, p) if j < h else p for j, p in enumerate(t)] for t, h in zip(tables, held)],
                shares=new, free=list(range(P - 1, u - 1, -1)), n_free=P - u, source=source, target=target)
