"""Measured cases of the paged key-value cache operators.

Three operators that a serving step runs one after the other:

* ``page_plan``: block tables and slot maps built on the GPU from request
  lengths. Request b is to hold ``ceil(lens[b] / page)`` pages: pages it no
  longer needs go back onto a stack of free pages, pages it lacks are taken
  from it, and every token row of the pass gets its cache slot and position.
* ``kv_append``: rotary embedding of the rows' queries and keys, and the rows'
  keys and values into their slots of the paged cache.
* ``paged_attention``: attention of each request's newest rows (one when
  decoding, several when verifying guesses) over its pages.

``run`` computes them either with elementary torch operations (``own`` false)
or through this package's calls (``own`` true).
"""

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def _pkg():
    import greedy_speculative_decoding_gb300 as pkg
    return pkg


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One verify pass of eight sequences (a pending token and eight
        # guesses each) between two rounds: a few pages change hands.
        dict(name="plan_verify_b8", op="plan", requests=8, lo=1024, hi=8192, rows=9, ragged=False, page=64, tight=False),
        # Decode step of a full server: one new token per request, some
        # requests finished since the last pass, small pages.
        dict(name="plan_decode_b512", op="plan", requests=512, lo=1, hi=8192, rows=1, ragged=False, page=16, tight=False),
        # Admission of a batch of prompts: every row of every prompt gets its
        # slot; the pool cannot take all of them.
        dict(name="plan_prompts_b250", op="plan", requests=250, lo=1, hi=4095, rows=0, ragged=False, page=16, tight=True),
        # A draft model's decode step: one row, straight from the fp32 projections.
        dict(name="append_draft_row", op="append", tokens=1, heads=14, kv_heads=2, head_dim=64, page=64, dtype="fp32",
             cache="bf16", context=512, rope=True, fused=False, pad=0),
        # Verify rows of eight sequences at the 14B shape, fp32 projections in
        # one fused q/k/v buffer.
        dict(name="append_verify_14b_b8", op="append", tokens=72, heads=40, kv_heads=8, head_dim=128, page=64,
             dtype="fp32", cache="bf16", context=8192, rope=True, fused=True, pad=8),
        # A long prompt's rows at the 7B shape, bf16 projections, small pages.
        dict(name="append_prompt_7b", op="append", tokens=16411, heads=28, kv_heads=4, head_dim=128, page=16,
             dtype="bf16", cache="bf16", context=16411, rope=True, fused=True, pad=0),
        # Draft decode step on its own: one token over a short cache.
        dict(name="attn_draft_512", op="attn", requests=1, lo=512, hi=512, rows=1, ragged=False, heads=14, kv_heads=2,
             head_dim=64, page=64, dtype="bf16", cache="bf16", tree=False, pad=0),
        # Plain decoding of a ragged batch at the 7B shape with small pages,
        # among them empty and just started requests.
        dict(name="attn_decode_7b_b32", op="attn", requests=32, lo=0, hi=8191, rows=1, ragged=False, heads=28,
             kv_heads=4, head_dim=128, page=16, dtype="bf16", cache="bf16", tree=False, pad=3),
        # Verify pass of one sequence at context 2048, fp32 queries as the
        # projections leave them.
        dict(name="attn_verify_7b_fp32", op="attn", requests=1, lo=2057, hi=2057, rows=9, ragged=False, heads=28,
             kv_heads=4, head_dim=128, page=64, dtype="fp32", cache="bf16", tree=False, pad=0),
        # Verify pass of eight sequences at the 14B shape, a different number
        # of guesses each.
        dict(name="attn_verify_14b_b8", op="attn", requests=8, lo=1024, hi=8192, rows=9, ragged=True, heads=40,
             kv_heads=8, head_dim=128, page=64, dtype="bf16", cache="bf16", tree=False, pad=7),
        # Guesses of a tree verified side by side at the draft's head layout, fp16.
        dict(name="attn_tree_fp16_b16", op="attn", requests=16, lo=5, hi=4099, rows=13, ragged=True, heads=14,
             kv_heads=2, head_dim=64, page=32, dtype="fp16", cache="fp16", tree=True, pad=0),
        # Decoding over long contexts at the 14B head layout: the largest.
        dict(name="attn_long_14b_b8", op="attn", requests=8, lo=65537, hi=131072, rows=1, ragged=False, heads=40,
             kv_heads=8, head_dim=128, page=128, dtype="bf16", cache="bf16", tree=False, pad=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "plan":
        requests = _log_int(rng, 1, 2000)
        rows = rng.choice([0, 1, rng.randint(2, 17)])
        hi = _log_int(rng, 1, 8192)
        if rows == 0:
            hi = max(1, min(hi, 500000 // requests))
        return dict(op="plan", requests=requests, lo=rng.randint(1, hi), hi=hi, rows=rows, ragged=rng.random() < 0.5,
                    page=page, tight=rng.random() < 0.3)
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8])
    head_dim = rng.choice([64, 128])
    if op == "append":
        tokens = _log_int(rng, 1, 16000)
        dtype = rng.choice(["fp32", "bf16", "fp16"])
        cache = dtype if dtype != "fp32" else rng.choice(["bf16", "fp16"])
        return dict(op="append", tokens=tokens, heads=min(heads, 32), kv_heads=kv_heads if heads <= 32 else 4,
                    head_dim=head_dim, page=page, dtype=dtype, cache=cache, context=_log_int(rng, 1, 32768),
                    rope=rng.random() < 0.8, fused=rng.random() < 0.5, pad=rng.choice([0, 0, rng.randint(1, 9)]))
    requests = _log_int(rng, 1, 128)
    rows = rng.choice([1, 1, rng.randint(2, 16)])
    tree = rows > 1 and rng.random() < 0.4
    # No more cache bytes and no more products than the largest listed case.
    most = min(131072, (8 * 98304 * 8 * 128) // (2 * requests * kv_heads * head_dim),
               4000000000 // (requests * rows * heads * head_dim))
    hi = _log_int(rng, 1, max(1, most))
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    return dict(op="attn", requests=requests, lo=rng.randint(0, hi), hi=hi, rows=rows, ragged=rows > 1 and rng.random() < 0.5,
                heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, dtype=dtype,
                cache="bf16" if dtype == "fp32" else dtype, tree=tree, pad=rng.choice([0, 0, rng.randint(1, 9)]))


def _lens_rows(case):
    """Length and newest rows of every request, in a fixed order (the seed
    permutes it): lengths spread evenly over lo..hi; rows 0 stands for the
    whole length (a prompt)."""
    n, lo, hi = case["requests"], case["lo"], case["hi"]
    lens = [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]
    if n == 1:
        lens = [hi]
    if case["rows"] == 0:
        rows = list(lens)
    elif case["ragged"]:
        rows = [min(lens[i], 1 + (i * 7) % case["rows"]) for i in range(n)]
    else:
        rows = [min(lens[i], case["rows"]) for i in range(n)]
    return lens, rows


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    if case["op"] == "plan":
        lens, rows = _lens_rows(case)
        page, n = case["page"], case["requests"]
        # lengths, row starts, held counts in and out, status; the table entry
        # of every page that a row lies in; slot and position of every row.
        entries = sum(_pages(a, page) - (a - r) // page for a, r in zip(lens, rows) if r)
        return {"bytes": 4 * (5 * n + entries + 2 * sum(rows)), "flops": 0}
    if case["op"] == "append":
        t, hd = case["tokens"], case["head_dim"]
        el = t * (case["heads"] + 2 * case["kv_heads"]) * hd
        nbytes = el * (_SIZE[case["dtype"]] + _SIZE[case["cache"]]) + 4 * t
        flops = 0
        if case["rope"]:
            nbytes += 4 * t + min(t, case["context"]) * hd * 4
            flops = 3 * t * (case["heads"] + case["kv_heads"]) * hd
        return {"bytes": nbytes, "flops": flops}
    lens, rows = _lens_rows(case)
    hd, page = case["head_dim"], case["page"]
    kv = sum(a for a, r in zip(lens, rows) if r) * case["kv_heads"] * hd * 2 * _SIZE[case["cache"]]
    n_rows = sum(rows)
    q = n_rows * case["heads"] * (2 * hd * _SIZE[case["dtype"]] + 4)
    tab = sum(_pages(a, page) for a in lens) * 4 + 8 * case["requests"]
    seen = sum(r * (a - r) + r * (r + 1) // 2 for a, r in zip(lens, rows))
    return {"bytes": kv + q + tab + (8 * n_rows if case["tree"] else 0), "flops": 4 * seen * case["heads"] * hd}


# ------------------------------------------------------------------ the inputs
def _i32(a):
    return torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()


def _prepare_plan(case, rs):
    """Requests between two passes: each holds the pages of its length before
    this pass; some finish (length 0 from now on) and some gave guesses back."""
    n, page = case["requests"], case["page"]
    lens, rows = (np.array(a, dtype=np.int64) for a in _lens_rows(case))
    order = rs.permutation(n)
    lens, rows = lens[order], rows[order]
    before = lens - rows
    if case["rows"]:
        before = before + rs.randint(0, 2 * case["rows"] + 1, n)   # the last pass's guesses, not all kept
        done = rs.random_sample(n) < 0.05
        done[0] = False
        lens, rows = np.where(done, 0, lens), np.where(done, 0, rows)
    held = (before + page - 1) // page
    need = (lens + page - 1) // page
    width = _pages(case["hi"] + 2 * case["rows"], page) + 3
    grow = int(np.maximum(need - held, 0).sum())
    n_free = 1 + (grow * 3 // 4 if case["tight"] else grow + 17)
    total = sum(2 * _pages(a + 2 * case["rows"], page) for a in _lens_rows(case)[0]) + 18   # the rest is in other hands
    perm = rs.permutation(total).astype(np.int32)
    tables = np.zeros((n, width), np.int32)
    at = 0
    for b in range(n):
        tables[b, :held[b]] = perm[at:at + held[b]]
        at += int(held[b])
    free = np.zeros(total, np.int32)
    free[:n_free] = perm[at:at + n_free]
    starts = np.concatenate([[0], np.cumsum(rows)])
    n_rows = sum(_lens_rows(case)[1]) + (5 if case["ragged"] else 0)   # a pass padded to a fixed number of rows
    return dict(case=case, lens=_i32(lens), starts=_i32(starts), tables=_i32(tables), held=_i32(held),
                free=_i32(free), n_free=_i32([n_free]), rows=n_rows,
                slots=torch.zeros(n_rows, dtype=torch.int32, device="cuda"),
                positions=torch.zeros(n_rows, dtype=torch.int32, device="cuda"),
                held_out=torch.zeros(n, dtype=torch.int32, device="cuda"),
                n_free_out=torch.zeros(1, dtype=torch.int32, device="cuda"),
                status=torch.zeros(n, dtype=torch.int32, device="cuda"))


def _randn(shape, dtype, gen, scale=1.0):
    t = torch.randn(shape, dtype=dtype, device="cuda", generator=gen)
    return t if scale == 1.0 else t.mul_(scale)


def _prepare_append(case, rs, gen):
    t, hd, page, pad = case["tokens"], case["head_dim"], case["page"], case["pad"]
    nq, nkv = case["heads"], case["kv_heads"]
    n = t + pad
    din, dc = _DT[case["dtype"]], _DT[case["cache"]]
    if case["fused"]:   # one buffer of projected rows, q | k | v side by side
        buf = _randn((n, (nq + 2 * nkv) * hd), din, gen)
        q, k, v = (x.view(n, -1, hd) for x in buf.split([nq * hd, nkv * hd, nkv * hd], dim=1))
    else:
        q, k, v = (_randn((n, h, hd), din, gen) for h in (nq, nkv, nkv))
    n_pages = _pages(t, page) + 3
    # Runs of consecutive tokens within scattered pages, as a table gives them.
    perm = rs.permutation(n_pages)[:_pages(t, page)]
    slots = (perm[:, None] * page + np.arange(page)[None]).reshape(-1)[:t]
    slots = np.concatenate([slots, np.full(pad, -1)])
    pos = np.concatenate([(rs.randint(0, case["context"]) + np.arange(t)) % case["context"], np.zeros(pad)])
    inv = 1.0e6 ** (-2.0 * np.arange(hd // 2) / hd)
    ang = np.arange(case["context"])[:, None] * inv[None]
    rope = torch.from_numpy(np.stack([np.cos(ang), np.sin(ang)], axis=-1).astype(np.float32)).cuda()
    st = dict(case=case, q=q, k=k, v=v, slots=_i32(slots), positions=_i32(pos), rope=rope if case["rope"] else None,
              k_cache=torch.zeros((n_pages, nkv, page, hd), dtype=dc, device="cuda"),
              v_cache=torch.zeros((n_pages, nkv, page, hd), dtype=dc, device="cuda"),
              q_out=torch.zeros((n, nq, hd), dtype=dc, device="cuda"))
    return st


def _prepare_attn(case, rs, gen):
    n, page, hd = case["requests"], case["page"], case["head_dim"]
    nq, nkv = case["heads"], case["kv_heads"]
    lens, rows = (np.array(a, dtype=np.int64) for a in _lens_rows(case))
    order = rs.permutation(n)
    lens, rows = lens[order], rows[order]
    held = (lens + page - 1) // page
    width = max(1, int(held.max()))
    n_pages = int(held.sum()) + 2
    perm = rs.permutation(n_pages).astype(np.int32)
    tables = np.zeros((n, width), np.int32)
    at = 0
    for b in range(n):
        tables[b, :held[b]] = perm[at:at + held[b]]
        at += int(held[b])
    starts = np.concatenate([[0], np.cumsum(rows)])
    t = int(starts[-1]) + case["pad"]
    t = max(t, 1)
    dq, dc = _DT[case["dtype"]], _DT[case["cache"]]
    # Keys and values in one pool, page by page, as a server lays them out.
    pool = _randn((n_pages, 2, nkv, page, hd), dc, gen)
    q = _randn((t, nq, hd), dq, gen, 2.0)
    mask = None
    if case["tree"]:   # row j sees itself and its ancestors among the pass's rows
        bits = np.zeros(t, np.int64)
        for b in range(n):
            s = int(starts[b])
            for j in range(int(rows[b])):
                bits[s + j] = 1 << j
                if j:
                    bits[s + j] |= bits[s + rs.randint(0, j)]
        mask = torch.from_numpy(bits).cuda()
    st = dict(case=case, q=q, k_cache=pool[:, 0], v_cache=pool[:, 1], tables=_i32(tables), lens=_i32(lens),
              starts=_i32(starts), max_rows=max(1, case["rows"]), mask=mask, scale=1.0 / math.sqrt(hd),
              out=torch.zeros((t, nq, hd), dtype=dq, device="cuda"),
              lse=torch.zeros((t, nq), dtype=torch.float32, device="cuda"), workspace=None)
    return st


def prepare(case, seed):
    rs = np.random.RandomState(seed % (2 ** 32))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "plan":
        return _prepare_plan(case, rs)
    if case["op"] == "append":
        return _prepare_append(case, rs, gen)
    st = _prepare_attn(case, rs, gen)
    if own:   # scratch that a serving loop keeps between its passes
        st["workspace"] = _pkg().paged_attention_workspace(st["q"], st["k_cache"], st["tables"], st["max_rows"])
    return st


# ------------------------------------------------------------------ plain forms
def _plain_plan(st):
    page = st["case"]["page"]
    lens, starts, tables, held, free = (st[x].long() for x in ("lens", "starts", "tables", "held", "free"))
    n_free = st["n_free"].long()
    n, width = tables.shape
    rows = starts[1:] - starts[:-1]
    need = (lens + page - 1) // page
    bad = (lens < 0) | (need > width) | (rows > lens)
    need = torch.where(bad, held, need)
    back, want = (held - need).clamp(min=0), (need - held).clamp(min=0)
    j = torch.arange(width, device=lens.device)[None]
    # Pages given back go on top of the stack, in request and table order.
    at = n_free + (back.cumsum(0) - back)[:, None] + j - need[:, None]
    m = (j >= need[:, None]) & (j < held[:, None])
    free[at[m]] = tables[m]
    top = n_free + back.sum()
    upto = want.cumsum(0)
    refused = (want > 0) & (upto > top)
    take = torch.where(refused, 0, want)
    # Page k of the pass comes from k places below the top.
    at = top - 1 - (upto - want)[:, None] - (j - held[:, None])
    m = (j >= held[:, None]) & (j < (held + take)[:, None])
    tables[m] = free[at[m]]
    st["tables"].copy_(tables)
    st["free"].copy_(free)
    st["held_out"].copy_(torch.where(refused | bad, held, need))
    st["n_free_out"].copy_(top - take.sum())
    st["status"].copy_(torch.where(bad, 2, refused.long()))
    row = torch.arange(st["rows"], device=lens.device)
    b = torch.searchsorted(starts[1:].contiguous(), row, right=True)
    live = (b < n) & (row >= starts[0])
    b = b.clamp(max=n - 1)
    live = live & ~(refused | bad)[b]
    pos = torch.where(live, lens[b] - starts[b + 1] + row, 0)
    slot = tables[b, pos // page] * page + pos % page
    st["slots"].copy_(torch.where(live, slot, -1))
    st["positions"].copy_(pos)
    return _plan_out(st)


def _plan_out(st):
    return {x: st[x] for x in ("tables", "held_out", "free", "n_free_out", "slots", "positions", "status")}


def _rotate(x, cs):
    half = x.shape[-1] // 2
    a, b = x[..., :half], x[..., half:]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat([a * c - b * s, b * c + a * s], dim=-1)


def _plain_append(st):
    page = st["case"]["page"]
    slots = st["slots"].long()
    live = slots >= 0
    q, k, v = (st[x][live].float() for x in ("q", "k", "v"))
    if st["rope"] is not None:
        cs = st["rope"][st["positions"].long()[live]]
        q, k = _rotate(q, cs), _rotate(k, cs)
    slots = slots[live]
    kc, vc = st["k_cache"], st["v_cache"]
    kc[slots // page, :, slots % page] = k.to(kc.dtype)
    vc[slots // page, :, slots % page] = v.to(vc.dtype)
    st["q_out"][live] = q.to(st["q_out"].dtype)
    return {"q": st["q_out"], "k_cache": kc, "v_cache": vc}


def _plain_attn(st):
    q, tables, lens, starts = st["q"], st["tables"].long(), st["lens"].long(), st["starts"].long()
    n, width = tables.shape
    t, nq, hd = q.shape
    _, nkv, page, _ = st["k_cache"].shape
    r = st["max_rows"]
    k, v = (st[x][tables].permute(0, 2, 1, 3, 4).reshape(n, nkv, width * page, hd).float()
            for x in ("k_cache", "v_cache"))
    j = torch.arange(r, device=q.device)
    rows = starts[1:] - starts[:-1]
    live = j[None] < rows[:, None]                                  # [n, r]
    at = (starts[:-1, None] + j[None]).clamp(max=t - 1)
    qp = q[at].float().view(n, r, nkv, nq // nkv, hd)
    slot = torch.arange(width * page, device=q.device)[None, None]  # [1, 1, s]
    first = (lens - rows)[:, None, None]
    if st["mask"] is None:
        seen = slot <= first + j[None, :, None]
    else:
        off = (slot - first).clamp(0, 63)
        seen = (slot < first) | (((st["mask"][at][:, :, None] >> off) & 1).bool() & (slot < first + 64))
    seen = seen & (slot < lens[:, None, None]) & live[:, :, None]
    s = torch.einsum("brhgd,bhsd->bhrgs", qp, k) * st["scale"]
    s = s.masked_fill(~seen[:, None, :, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m.clamp(min=-3.0e38))
    l = p.sum(-1, keepdim=True)
    o = torch.einsum("bhrgs,bhsd->bhrgd", p, v) / torch.where(l > 0, l, 1.0)
    o = o.permute(0, 2, 1, 3, 4).reshape(n, r, nq, hd)
    lse = (m + torch.log(l))[..., 0].permute(0, 2, 1, 3).reshape(n, r, nq)
    st["out"][at[live]] = o[live].to(q.dtype)
    st["lse"][at[live]] = lse[live]
    return {"out": st["out"], "lse": st["lse"]}


# ------------------------------------------------------------------ one pass
def run(state):
    st = state
    op = st["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}[op](st)
    pkg = _pkg()
    if op == "plan":
        pkg.page_plan(st["lens"], st["starts"], st["tables"], st["held"], st["free"], st["n_free"], st["case"]["page"],
                      slots=st["slots"], positions=st["positions"], held_out=st["held_out"],
                      n_free_out=st["n_free_out"], status=st["status"])
        return _plan_out(st)
    if op == "append":
        pkg.kv_append(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"], q=st["q"], q_out=st["q_out"],
                      positions=st["positions"], rope=st["rope"])
        return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    pkg.paged_attention(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], starts=st["starts"],
                        max_rows=st["max_rows"], mask=st["mask"], scale=st["scale"], out=st["out"], lse=st["lse"],
                        workspace=st["workspace"])
    return {"out": st["out"], "lse": st["lse"]}


# ------------------------------------------------------------------ in 64 bits
def _exact_plan(st):
    page = st["case"]["page"]
    a = {x: st[x].cpu().numpy().astype(np.int64) for x in ("lens", "starts", "tables", "held", "free", "n_free")}
    tables, free, held = a["tables"].copy(), a["free"].copy(), a["held"].copy()
    n, width = tables.shape
    need = -(-a["lens"] // page)
    status = np.zeros(n, np.int64)
    top = int(a["n_free"][0])
    for b in range(n):
        if a["lens"][b] < 0 or need[b] > width or a["starts"][b + 1] - a["starts"][b] > a["lens"][b]:
            status[b] = 2
            continue
        back = held[b] - need[b]
        if back > 0:
            free[top:top + back] = tables[b, need[b]:held[b]]
            top += int(back)
            held[b] = need[b]
    short = False
    for b in range(n):
        want = int(need[b] - held[b])
        if status[b] or want <= 0:
            continue
        short = short or want > top
        if short:
            status[b] = 1
            continue
        tables[b, held[b]:need[b]] = free[top - want:top][::-1]
        top -= want
        held[b] = need[b]
    slots, pos = np.full(st["rows"], -1, np.int64), np.zeros(st["rows"], np.int64)
    for b in range(n):
        s, e = int(a["starts"][b]), int(a["starts"][b + 1])
        if status[b] or e <= s:
            continue
        pos[s:e] = a["lens"][b] - (e - s) + np.arange(e - s)
        slots[s:e] = tables[b, pos[s:e] // page] * page + pos[s:e] % page
    res = dict(tables=tables, held_out=held, free=free, n_free_out=np.array([top]), slots=slots, positions=pos,
               status=status)
    return {x: torch.from_numpy(res[x].astype(np.int32)).cuda() for x in res}


def _exact_append(st):
    page, hd = st["case"]["page"], st["case"]["head_dim"]
    half = hd // 2
    out = {"q": st["q_out"].double(), "k_cache": st["k_cache"].double(), "v_cache": st["v_cache"].double()}
    rows = torch.nonzero(st["slots"] >= 0)[:, 0]
    slot = st["slots"].long()[rows]

    def turned(x):
        x = x[rows].double()
        if st["rope"] is None:
            return x
        z = torch.view_as_complex(st["rope"].double()[st["positions"].long()[rows]].contiguous())[:, None]
        w = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * z
        return torch.cat([w.real, w.imag], dim=-1)

    page_of, off = torch.div(slot, page, rounding_mode="floor"), slot.remainder(page)
    out["q"][rows] = turned(st["q"])
    out["k_cache"].transpose(1, 2)[page_of, off] = turned(st["k"])
    out["v_cache"].transpose(1, 2)[page_of, off] = st["v"][rows].double()
    return out


def _exact_attn(st):
    nq, hd = st["q"].shape[1:]
    _, nkv, page, _ = st["k_cache"].shape
    g = nq // nkv
    out, lse = st["out"].double(), st["lse"].double()
    lens, starts = st["lens"].tolist(), st["starts"].tolist()
    bits = None if st["mask"] is None else st["mask"].tolist()
    for b, n in enumerate(lens):
        s, e = starts[b], starts[b + 1]
        if e <= s:
            continue
        ids = st["tables"][b, :_pages(n, page)].long()
        for h in range(nkv):
            k = st["k_cache"][ids, h].reshape(-1, hd)[:n].double()
            v = st["v_cache"][ids, h].reshape(-1, hd)[:n].double()
            for i in range(s, e):
                first, j = n - (e - s), i - s
                see = torch.zeros(n, dtype=torch.bool)
                see[:first] = True
                for c in range(e - s):
                    see[first + c] = c <= j if bits is None else bool(bits[i] >> c & 1)
                x = (st["q"][i, h * g:(h + 1) * g].double() @ k.t()) * st["scale"]
                x[:, ~see.cuda()] = float("-inf")
                lse[i, h * g:(h + 1) * g] = torch.logsumexp(x, dim=-1)
                out[i, h * g:(h + 1) * g] = torch.softmax(x, dim=-1) @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "attn":
        lens, rows = _lens_rows(case)
        if sum(rows) * case["kv_heads"] > 8000:
            return None
    st = prepare(case, seed)
    return {"plan": _exact_plan, "append": _exact_append, "attn": _exact_attn}[case["op"]](st)
