"""Measured cases of prompt chunks over a paged cache, of pages that several
requests hold, and of token log probabilities.

* ``chunk``: attention of a chunk of new tokens (whole prompts or pieces of
  them) over a key-value cache in pages (``chunk_attention``).
* ``branch``: a step in which some continuations end and others are forked in
  their place: pages released (``page_free``), tables shared and the partly
  filled last pages given out anew (``page_fork``), those pages copied in every
  layer (``page_copy``).
* ``compact``: the held pages move to the lowest numbers (``page_compact``),
  with their contents in every layer (``page_copy``).
* ``logprobs``: log probabilities of given tokens, entropy, rank and the top
  alternatives of rows of logits (``token_logprobs``).

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
        # A short prompt at the 0.5B draft's head layout: one call, latency.
        dict(name="chunk_draft_prompt", op="chunk", requests=1, lo=97, hi=97, rows=97, ragged=False, heads=14,
             kv_heads=2, head_dim=64, page=16, dtype="fp16", pad=0),
        # A 512-token prompt's second half as the 7B projections leave it: fp32 queries.
        dict(name="chunk_half_7b_fp32", op="chunk", requests=1, lo=512, hi=512, rows=256, ragged=False, heads=28,
             kv_heads=4, head_dim=128, page=64, dtype="fp32", pad=0),
        # Whole prompts of different lengths admitted together at the 7B shape.
        dict(name="chunk_prompts_7b_b9", op="chunk", requests=9, lo=33, hi=4099, rows=4099, ragged=False, heads=28,
             kv_heads=4, head_dim=128, page=64, dtype="bf16", pad=5),
        # Chunks of different lengths behind contexts of different lengths, fp16, small pages.
        dict(name="chunk_ragged_fp16_b8", op="chunk", requests=8, lo=1500, hi=8192, rows=700, ragged=True, heads=14,
             kv_heads=2, head_dim=64, page=16, dtype="fp16", pad=0),
        # A long prompt's last chunk at the 14B head layout: the largest.
        dict(name="chunk_long_14b", op="chunk", requests=1, lo=32768, hi=32768, rows=2048, ragged=False, heads=40,
             kv_heads=8, head_dim=128, page=128, dtype="bf16", pad=0),
        # Four continuations of a short prompt, two of them replaced, in a draft model's cache.
        dict(name="branch_draft_b4", op="branch", requests=4, forks=2, lo=200, hi=700, page=64, layers=24, kv_heads=2,
             head_dim=64, dtype="bf16"),
        # Every second of 256 continuations at the 7B shape replaced, small pages.
        dict(name="branch_7b_b256", op="branch", requests=256, forks=128, lo=500, hi=8000, page=16, layers=28,
             kv_heads=4, head_dim=128, dtype="bf16"),
        # A small draft cache with holes, packed.
        dict(name="compact_draft", op="compact", requests=8, lo=30, hi=900, page=64, layers=24, kv_heads=2, head_dim=64,
             dtype="fp16", spare=0.5),
        # A server's cache after hours of requests coming and going, one layer group of the 7B shape.
        dict(name="compact_7b_b200", op="compact", requests=200, lo=1, hi=4000, page=16, layers=7, kv_heads=4,
             head_dim=128, dtype="bf16", spare=1.0),
        # One decoded token of a sequence with its five top alternatives, logits as the LM head leaves them.
        dict(name="logprobs_row", op="logprobs", rows=1, vocab=151936, dtype="fp32", top=5, masked=0.0, pad=0),
        # A verify pass of eight sequences at the 14B shape, nine rows each.
        dict(name="logprobs_verify_b8", op="logprobs", rows=72, vocab=152064, dtype="fp32", top=20, masked=0.0, pad=0),
        # A prompt's tokens scored from 16-bit logits, some of the vocabulary masked, rows of odd length.
        dict(name="logprobs_prompt", op="logprobs", rows=1021, vocab=151665, dtype="bf16", top=1, masked=0.1, pad=3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "branch", "compact", "logprobs"])
    page = rng.choice([16, 32, 64, 128, 256])
    head_dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "chunk":
        heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8])
        requests = _log_int(rng, 1, 24)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        # No more products than the largest listed case, 64 times fewer in fp32.
        most = 2048 * 32768 * 40 * 128 // (64 if dtype == "fp32" else 1) // (requests * heads * head_dim)
        hi = _log_int(rng, 64, min(32768, max(64, most)))
        rows = _log_int(rng, 1, max(1, min(hi, 4096, most // hi)))
        return dict(op="chunk", requests=requests, lo=rng.randint(0, hi), hi=hi, rows=rows, ragged=rng.random() < 0.5,
                    heads=heads, kv_heads=kv_heads, head_dim=head_dim, page=page, dtype=dtype,
                    pad=rng.choice([0, 0, rng.randint(1, 9)]))
    layers = rng.choice([1, 2, 24, 28])
    if op == "branch":
        requests = _log_int(rng, 2, 400)
        forks = rng.randint(1, requests - 1)
        hi = _log_int(rng, 1, min(32768, 2000000 // requests))
        # The cache of all requests, within a few GB.
        layers = max(1, min(layers, 4000000000 // (4 * kv_heads * head_dim * (requests * (hi + 2 * page)))))
        return dict(op="branch", requests=requests, forks=forks, lo=rng.randint(0, hi), hi=hi, page=page, layers=layers,
                    kv_heads=kv_heads, head_dim=head_dim, dtype=rng.choice(["bf16", "fp16"]))
    if op == "compact":
        requests = _log_int(rng, 1, 400)
        hi = _log_int(rng, 1, min(16384, 400000 // requests))
        spare = rng.choice([0.1, 0.5, 1.0, 3.0])
        layers = max(1, min(layers, int(4.0e9 / ((1 + spare) * 4 * kv_heads * head_dim * (requests * (hi + page))))))
        return dict(op="compact", requests=requests, lo=rng.randint(0, hi), hi=hi, page=page, layers=layers,
                    kv_heads=kv_heads, head_dim=head_dim, dtype=rng.choice(["bf16", "fp16"]), spare=spare)
    vocab = rng.choice([1024, _log_int(rng, 2, 200000), 151936, 152064, rng.randint(100000, 260000)])
    dtype = rng.choice(["fp32", "fp32", "bf16", "fp16"])
    rows = _log_int(rng, 1, max(1, min(4096, 150000000 // vocab)))
    return dict(op="logprobs", rows=rows, vocab=vocab, dtype=dtype, top=min(vocab, rng.choice([0, 1, 5, 20, 32])),
                masked=rng.choice([0.0, 0.0, 0.1, 0.9]), pad=rng.choice([0, 0, rng.randint(1, 9)]))


def _lens(case):
    """Lengths of the requests, spread evenly over lo..hi (the seed permutes them)."""
    n, lo, hi = case["requests"], case["lo"], case["hi"]
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lens_rows(case):
    """Length and new rows of every request, in a fixed order."""
    lens = _lens(case)
    if case["ragged"]:
        rows = [min(a, 1 + (case["rows"] - 1) * ((5 * i + 3) % 8 + 1) // 8) for i, a in enumerate(lens)]
    else:
        rows = [min(a, case["rows"]) for a in lens]
    return lens, rows


def _pages(tokens, page):
    return -(-tokens // page)


def _slot_bytes(case):
    """Keys and values of one slot in every layer."""
    return 2 * case["layers"] * case["kv_heads"] * case["head_dim"] * _SIZE[case["dtype"]]


def _fork_lens(case):
    """Tokens of the sources of a branch step: the first requests, in turn."""
    lens, stay = _lens(case), case["requests"] - case["forks"]
    return [lens[i % stay] for i in range(case["forks"])]


def work(case):
    if case["op"] == "chunk":
        lens, rows = _lens_rows(case)
        hd, cache = case["head_dim"], 2
        kv = sum(a for a, r in zip(lens, rows) if r) * case["kv_heads"] * hd * 2 * cache
        n_rows = sum(rows)
        q = n_rows * case["heads"] * (2 * hd * _SIZE[case["dtype"]] + 4)
        tab = sum(_pages(a, case["page"]) for a in lens) * 4 + 8 * case["requests"]
        seen = sum(r * (a - r) + r * (r + 1) // 2 for a, r in zip(lens, rows))
        return {"bytes": kv + q + tab, "flops": 4 * seen * case["heads"] * hd}
    page = case.get("page")
    if case["op"] == "branch":
        # Released and shared: a table entry and a page's count, each read and
        # written; the copied slots.
        lens = _fork_lens(case)
        entries = sum(_pages(a, page) for a in lens)
        return {"bytes": 2 * _slot_bytes(case) * sum(a % page for a in lens) + 4 * 4 * entries + 40 * case["forks"],
                "flops": 0}
    if case["op"] == "compact":
        # Every entry and count read, the moved entries, counts and pages
        # written, the stack of free pages written. Of the held pages the share
        # above their number moves (the same for every seed, within a few).
        held = sum(_pages(a, page) for a in _lens(case))
        total = held + int(case["spare"] * held) + 1
        moved = held * (total - held) // total
        return {"bytes": moved * page * 2 * _slot_bytes(case) + 4 * (held + moved) + 4 * (held + 3 * moved)
                + 4 * (total - held), "flops": 0}
    n, k = case["rows"], case["top"]
    return {"bytes": n * case["vocab"] * _SIZE[case["dtype"]] + n * (16 + 8 * k), "flops": 6 * n * case["vocab"]}


# ------------------------------------------------------------------ the inputs
def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


def _randn(shape, dtype, gen, scale=1.0):
    t = torch.randn(shape, dtype=dtype, device="cuda", generator=gen)
    return t if scale == 1.0 else t.mul_(scale)


def _prepare_chunk(case, rs, gen):
    n, page, hd = case["requests"], case["page"], case["head_dim"]
    nq, nkv = case["heads"], case["kv_heads"]
    lens, rows = (np.array(a, dtype=np.int64) for a in _lens_rows(case))
    order = rs.permutation(n)
    lens, rows = lens[order], rows[order]
    held = (lens + page - 1) // page
    n_pages = int(held.sum()) + 2
    perm = rs.permutation(n_pages).astype(np.int32)
    tables = np.zeros((n, max(1, int(held.max()))), np.int32)
    at = 0
    for b in range(n):
        tables[b, :held[b]] = perm[at:at + held[b]]
        at += int(held[b])
    starts = np.concatenate([[0], np.cumsum(rows)])
    t = max(1, int(starts[-1]) + case["pad"])
    dq = _DT[case["dtype"]]
    dc = torch.bfloat16 if case["dtype"] == "fp32" else dq
    # Keys and values in one pool, page by page, as a server lays them out.
    pool = _randn((n_pages, 2, nkv, page, hd), dc, gen)
    sizes = [(int(a), int(s), int(s + r)) for a, s, r in zip(lens, starts, rows)]
    return dict(case=case, sizes=sizes, q=_randn((t, nq, hd), dq, gen, 2.0), k_cache=pool[:, 0], v_cache=pool[:, 1],
                tables=_i32(tables), lens=_i32(lens), starts=_i32(starts), max_rows=max(1, int(rows.max())),
                scale=1.0 / math.sqrt(hd), out=torch.zeros((t, nq, hd), dtype=dq, device="cuda"),
                lse=torch.zeros((t, nq), dtype=torch.float32, device="cuda"), workspace=None)


def _pool(case, n_pages, gen):
    """A cache of all layers: [layers, keys and values, pages, heads, page, head_dim]."""
    shape = (case["layers"], 2, n_pages, case["kv_heads"], case["page"], case["head_dim"])
    pool = torch.empty(shape, dtype=_DT[case["dtype"]], device="cuda")
    for layer in range(case["layers"]):
        pool[layer].normal_(generator=gen)
    return pool


def _prepare_branch(case, rs, gen):
    """Continuations as the same step has left them once before: request
    stay + i is a fork of request i % stay. They end, last first, and are
    forked anew; the tables, counts and stack come out as they went in."""
    n, forks, page = case["requests"], case["forks"], case["page"]
    stay = n - forks
    lens = np.array(_lens(case), np.int64)
    src = np.arange(forks) % stay
    order = rs.permutation(n)                 # where in the batch each request sits
    lens[stay:] = lens[src]
    width = max(1, int(_pages(int(lens.max()), page))) + 1
    own_pages = (lens[:stay] + page - 1) // page
    n_pages = int(own_pages.sum()) + forks + 5
    perm = rs.permutation(n_pages).astype(np.int32)
    tables, held, shares = np.zeros((n, width), np.int32), np.zeros(n, np.int64), np.zeros(n_pages, np.int32)
    at = 0
    for b in range(stay):
        held[b] = own_pages[b]
        tables[b, :held[b]] = perm[at:at + held[b]]
        at += int(held[b])
    for i in range(forks):
        s, d = src[i], stay + i
        held[d] = held[s]
        full = int(lens[s]) // page
        tables[d, :full] = tables[s, :full]
        shares[tables[s, :full]] += 1
        if held[s] > full:
            tables[d, full] = perm[at]
            at += 1
    free = np.zeros(n_pages, np.int32)
    free[:n_pages - at] = perm[at:]
    at_row = np.argsort(order)                # request r lies in row at_row[r]
    rows = np.argsort(at_row)
    pool = _pool(case, n_pages, gen)
    z = lambda m: torch.zeros(m, dtype=torch.int32, device="cuda")
    return dict(case=case, tables=_i32(tables[rows]), held=_i32(held[rows]), lens=_i32(lens[rows]), shares=_i32(shares),
                free=_i32(free), n_free=_i32([n_pages - at]), ended=_i32(at_row[stay:][::-1]), keep=z(forks),
                src=_i32(at_row[src]), dst=_i32(at_row[stay:]), source=z(forks), target=z(forks), slots=z(forks),
                status=z(forks), free_status=z(forks), k_cache=pool[:, 0], v_cache=pool[:, 1])


def _prepare_compact(case, rs, gen):
    n, page = case["requests"], case["page"]
    lens = np.array(_lens(case), np.int64)[rs.permutation(n)]
    held = (lens + page - 1) // page
    total = int(held.sum())
    n_pages = total + int(case["spare"] * total) + 1
    perm = rs.permutation(n_pages).astype(np.int32)
    tables, shares = np.full((n, max(1, int(held.max())) + 1), -1, np.int32), np.zeros(n_pages, np.int32)
    at = 0
    for b in range(n):
        tables[b, :held[b]] = perm[at:at + held[b]]
        at += int(held[b])
        if b % 4 == 3:                        # the first pages are a prefix that another request holds too
            k = int(min(held[b], held[b - 1]) // 2)
            tables[b, :k] = tables[b - 1, :k]
            shares[tables[b, :k]] += 1
    pool = _pool(case, n_pages, gen)
    z = lambda m: torch.zeros(m, dtype=torch.int32, device="cuda")
    t = _i32(tables)
    return dict(case=case, tables=t, held=_i32(held), shares=_i32(shares), tables_out=torch.zeros_like(t),
                shares_out=z(n_pages), free=z(n_pages), n_free=z(1), source=z(n_pages // 2), target=z(n_pages // 2),
                count=z(1), k_cache=pool[:, 0], v_cache=pool[:, 1])


def _prepare_logprobs(case, rs, gen):
    n, vocab = case["rows"] + case["pad"], case["vocab"]
    dt = _DT[case["dtype"]]
    logits = torch.empty((n, vocab), dtype=dt, device="cuda")
    # A broad bulk and a row's own sharpness: some rows nearly certain, some open.
    sharp = torch.from_numpy(np.exp(rs.uniform(0.0, 1.5, (n, 1))).astype(np.float32)).cuda()
    for i in range(0, n, 256):
        m = min(256, n - i)
        logits[i:i + m] = torch.randn((m, vocab), device="cuda", generator=gen).mul_(sharp[i:i + m]).to(dt)
    tokens = rs.randint(0, vocab, n)
    if case["masked"]:                        # a grammar leaves part of the vocabulary
        gone = torch.rand(vocab, device="cuda", generator=gen) < case["masked"]
        gone[0] = False
        logits.masked_fill_(gone, float("-inf"))
        tokens = np.where(gone.cpu().numpy()[tokens], 0, tokens)
    tokens[case["rows"]:] = -1                # a batch padded to a fixed number of rows
    k = case["top"]
    z = lambda *m, dtype=torch.float32: torch.zeros(m, dtype=dtype, device="cuda")
    return dict(case=case, logits=logits, tokens=_i32(tokens), logprob=z(n), entropy=z(n), rank=z(n, dtype=torch.int32),
                top_ids=z(n, k, dtype=torch.int32), top_logprobs=z(n, k))


_PREPARE = {"chunk": _prepare_chunk, "branch": _prepare_branch, "compact": _prepare_compact,
            "logprobs": _prepare_logprobs}


def prepare(case, seed):
    rs = np.random.RandomState(seed % (2 ** 32))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = _PREPARE[case["op"]](case, rs, gen)
    if own and case["op"] == "chunk":   # scratch that a serving loop keeps between its passes
        st["workspace"] = _pkg().chunk_attention_workspace(st["q"], st["k_cache"], st["tables"], st["max_rows"])
    return st


# ------------------------------------------------------------------ plain forms
def _plain_chunk(st):
    q, tables = st["q"], st["tables"].long()
    nq, hd = q.shape[1:]
    _, nkv, page, _ = st["k_cache"].shape
    g = nq // nkv
    for b, (n, s, e) in enumerate(st["sizes"]):   # (known on the host, where the batch is put together)
        r = e - s
        if r <= 0:
            continue
        ids = tables[b, :_pages(n, page)]
        pos = torch.arange(n - r, n, device=q.device)[:, None]
        unseen = torch.arange(n, device=q.device)[None] > pos          # [r, n]
        for h in range(nkv):
            k = st["k_cache"][ids, h].reshape(-1, hd)[:n].float()
            v = st["v_cache"][ids, h].reshape(-1, hd)[:n].float()
            x = torch.matmul(q[s:e, h * g:(h + 1) * g].float().transpose(0, 1), k.t()).mul_(st["scale"])   # [g, r, n]
            x.masked_fill_(unseen[None], float("-inf"))
            m = x.amax(-1, keepdim=True)
            x.sub_(m).exp_()
            l = x.sum(-1, keepdim=True)
            o = torch.matmul(x, v) / l
            st["out"][s:e, h * g:(h + 1) * g] = o.transpose(0, 1).to(q.dtype)
            st["lse"][s:e, h * g:(h + 1) * g] = (m + torch.log(l))[..., 0].t()
    return {"out": st["out"], "lse": st["lse"]}


def _copy_pages(st, source, target, slots=None):
    """Pages source into pages target of every layer, or their first slots."""
    page = st["case"]["page"]
    for cache in (st["k_cache"], st["v_cache"]):
        new = cache[:, source]
        if slots is not None:
            off = torch.arange(page, device=source.device)
            new = torch.where((off[None] < slots[:, None])[None, :, None, :, None], new, cache[:, target])
        cache[:, target] = new


def _plain_branch(st):
    page = st["case"]["page"]
    tables, held, shares, free, lens = (st[x].long() for x in ("tables", "held", "shares", "free", "lens"))
    ended, keep, src, dst = (st[x].long() for x in ("ended", "keep", "src", "dst"))
    width = tables.shape[1]
    j = torch.arange(width, device=held.device)[None]
    # Release: pages whose last holder goes, each at its first place in the list.
    first = (keep + page - 1) // page
    gone = (j >= first[:, None]) & (j < held[ended][:, None])
    pages = tables[ended][gone]
    times = torch.zeros_like(shares).index_add_(0, pages, torch.ones_like(pages))
    at = torch.full_like(shares, pages.numel()).scatter_reduce_(0, pages, torch.arange(pages.numel(), device=held.device),
                                                                "amin")
    back = pages[(times[pages] > shares[pages]) & (at[pages] == torch.arange(pages.numel(), device=held.device))]
    shares = (shares - times).clamp(min=0)
    n_free = st["n_free"].long()
    where = n_free + torch.arange(back.numel(), device=held.device)
    free[where] = back
    n_free = n_free + back.numel()
    held[ended] = first
    st["free_status"].zero_()
    # Fork: shared pages, and a new one for the slots of a partly filled one.
    n = lens[src]
    full, part = n // page, n % page
    want = (part > 0).long()
    before = want.cumsum(0) - want
    sharing = j < full[:, None]
    entries = torch.where(sharing, tables[src], tables[dst])
    shares.index_add_(0, tables[src][sharing], torch.ones_like(tables[src][sharing]))
    new = free[(n_free - 1 - before).clamp(min=0)]
    source = torch.where(want > 0, tables[src].gather(1, full[:, None].clamp(max=width - 1))[:, 0], -1)
    target = torch.where(want > 0, new, -1)
    entries = torch.where((j == full[:, None]) & (want > 0)[:, None], new[:, None], entries)
    tables[dst] = entries
    held[dst] = full + want
    n_free = n_free - want.sum()
    for name, x in dict(tables=tables, held=held, shares=shares, free=free, n_free=n_free, source=source, target=target,
                        slots=part).items():
        st[name].copy_(x)
    st["status"].zero_()
    m = want > 0
    _copy_pages(st, source[m], target[m], part[m])
    return _branch_out(st)


def _branch_out(st):
    return {x: st[x] for x in ("tables", "held", "shares", "free", "n_free", "source", "target", "slots", "status",
                               "free_status", "k_cache", "v_cache")}


def _plain_compact(st):
    tables, held, shares = st["tables"].long(), st["held"].long(), st["shares"]
    n_pages = shares.shape[0]
    used = torch.zeros(n_pages, dtype=torch.bool, device=shares.device)
    live = torch.arange(tables.shape[1], device=held.device)[None] < held[:, None]
    used[tables[live]] = True
    number = torch.arange(n_pages, device=shares.device)
    low = number < used.sum()
    source, target = number[used & ~low], number[~used & low]
    to = number.clone()
    to[source] = target
    st["tables_out"].copy_(torch.where(live, to[tables.clamp(min=0)], tables))
    new = torch.where(used, shares, 0)
    new[target] = shares[source]
    new[source] = 0
    st["shares_out"].copy_(new)
    n_free = n_pages - used.sum()
    st["free"].copy_(torch.where(number < n_free, n_pages - 1 - number, st["free"]))
    st["n_free"].copy_(n_free)
    m = source.numel()
    for name, x in (("source", source), ("target", target)):
        st[name].fill_(-1)
        st[name][:m] = x.int()
    st["count"].fill_(m)
    _copy_pages(st, source, target)
    return _compact_out(st)


def _compact_out(st):
    return {x: st[x] for x in ("tables_out", "shares_out", "free", "n_free", "source", "target", "count", "k_cache",
                               "v_cache")}


def _plain_logprobs(st):
    k = st["case"]["top"]
    rows = torch.nonzero(st["tokens"] >= 0)[:, 0]
    t = st["tokens"][rows].long()
    n, vocab = rows.numel(), st["logits"].shape[1]
    number = torch.arange(vocab, device=t.device)
    for i in range(0, n, 512):
        r, tok = rows[i:i + 512], t[i:i + 512, None]
        x = st["logits"][r].float()
        m = x.amax(-1, keepdim=True)
        d = x - m
        e = torch.exp(d)
        s = e.sum(-1, keepdim=True)
        mean = torch.where(e > 0, e * d, 0.0).sum(-1, keepdim=True) / s
        logs = torch.log(s)
        mine = x.gather(1, tok)
        st["logprob"][r] = (mine - m - logs)[:, 0]
        st["entropy"][r] = (logs - mean)[:, 0]
        st["rank"][r] = ((x > mine) | ((x == mine) & (number[None] < tok))).sum(-1).int()
        if k:
            # Order by value, then by number: one whole number for both.
            bits = (x + 0.0).view(torch.int32)
            key = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long() * (1 << 32) - number[None]
            ids = -(torch.topk(key, k, dim=-1).values) % (1 << 32)
            st["top_ids"][r] = ids.int()
            st["top_logprobs"][r] = x.gather(1, ids) - m - logs
    return _logprobs_out(st)


def _logprobs_out(st):
    return {x: st[x] for x in ("logprob", "entropy", "rank", "top_ids", "top_logprobs")}


# ------------------------------------------------------------------ one pass
_PLAIN = {"chunk": _plain_chunk, "branch": _plain_branch, "compact": _plain_compact, "logprobs": _plain_logprobs}


def run(state):
    st = state
    op = st["case"]["op"]
    if not own:
        return _PLAIN[op](st)
    pkg = _pkg()
    if op == "chunk":
        pkg.chunk_attention(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], starts=st["starts"],
                            max_rows=st["max_rows"], scale=st["scale"], out=st["out"], lse=st["lse"],
                            workspace=st["workspace"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "branch":
        page = st["case"]["page"]
        pkg.page_free(st["ended"], st["tables"], st["held"], st["shares"], st["free"], st["n_free"], page,
                      keep=st["keep"], status=st["free_status"])
        pkg.page_fork(st["src"], st["dst"], st["lens"], st["tables"], st["held"], st["shares"], st["free"],
                      st["n_free"], page, source=st["source"], target=st["target"], slots=st["slots"],
                      status=st["status"])
        pkg.page_copy(st["source"], st["target"], st["k_cache"], st["v_cache"], slots=st["slots"])
        return _branch_out(st)
    if op == "compact":
        pkg.page_compact(st["tables"], st["held"], st["shares"], st["free"], st["n_free"], tables_out=st["tables_out"],
                         shares_out=st["shares_out"], source=st["source"], target=st["target"], count=st["count"])
        pkg.page_copy(st["source"], st["target"], st["k_cache"], st["v_cache"], count=st["count"])
        return _compact_out(st)
    pkg.token_logprobs(st["logits"], st["tokens"], top=st["case"]["top"], logprob=st["logprob"], entropy=st["entropy"],
                       rank=st["rank"], top_ids=st["top_ids"], top_logprobs=st["top_logprobs"])
    return _logprobs_out(st)


# ------------------------------------------------------------------ in 64 bits
def _exact_chunk(st):
    nq, hd = st["q"].shape[1:]
    _, nkv, page, _ = st["k_cache"].shape
    g = nq // nkv
    out, lse = st["out"].double(), st["lse"].double()
    lens, starts = st["lens"].tolist(), st["starts"].tolist()
    for b, n in enumerate(lens):
        slots = [int(p) for p in st["tables"][b, :_pages(n, page)]]
        for i in range(starts[b], starts[b + 1], 256):          # a few rows at a time, each cut to what it sees
            e = min(i + 256, starts[b + 1])
            last = n - (starts[b + 1] - e)                      # slots that row e - 1 sees
            seen = torch.ones((e - i, last), dtype=torch.bool, device="cuda").tril(last - (e - i))
            for h in range(nq):
                k, v = (torch.cat([st[x][p, h // g] for p in slots])[:last].double() for x in ("k_cache", "v_cache"))
                x = st["scale"] * (st["q"][i:e, h].double() @ k.t())
                x = torch.where(seen, x, float("-inf"))
                lse[i:e, h] = torch.logsumexp(x, dim=-1)
                out[i:e, h] = torch.softmax(x, dim=-1) @ v
    return {"out": out, "lse": lse}


def _lists(st, names):
    return {x: st[x].cpu().tolist() for x in names}


def _exact_branch(st):
    page = st["case"]["page"]
    a = _lists(st, ("tables", "held", "shares", "free", "n_free", "lens", "ended", "keep", "src", "dst"))
    tables, held, shares, free, top = a["tables"], a["held"], a["shares"], a["free"], a["n_free"][0]
    holders = [s + 1 for s in shares]
    released = []
    for b, keep in zip(a["ended"], a["keep"]):
        for x in range(_pages(keep, page), held[b]):
            holders[tables[b][x]] -= 1
            released.append(tables[b][x])
        held[b] = _pages(keep, page)
    done = set()
    for p in released:
        if holders[p] == 0 and p not in done:
            done.add(p)
            free[top] = p
            top += 1
    shares = [max(h - 1, 0) for h in holders]
    source, target, slots = [], [], []
    k, v = st["k_cache"].clone(), st["v_cache"].clone()
    for s, d in zip(a["src"], a["dst"]):
        n = a["lens"][s]
        for x in range(n // page):
            tables[d][x] = tables[s][x]
            shares[tables[s][x]] += 1
        held[d] = _pages(n, page)
        slots.append(n % page)
        if n % page:
            top -= 1
            source.append(tables[s][n // page])
            target.append(free[top])
            tables[d][n // page] = free[top]
            k[:, target[-1], :, :n % page] = st["k_cache"][:, source[-1], :, :n % page]
            v[:, target[-1], :, :n % page] = st["v_cache"][:, source[-1], :, :n % page]
        else:
            source.append(-1)
            target.append(-1)
    res = dict(tables=tables, held=held, shares=shares, free=free, n_free=[top], source=source, target=target,
               slots=slots, status=[0] * len(slots), free_status=[0] * len(slots))
    return {**{x: _i32(y) for x, y in res.items()}, "k_cache": k, "v_cache": v}


def _exact_compact(st):
    a = _lists(st, ("tables", "held", "shares"))
    n_pages = len(a["shares"])
    held = sorted({p for row, h in zip(a["tables"], a["held"]) for p in row[:h]})
    u = len(held)
    source = [p for p in held if p >= u]
    target = sorted(set(range(u)) - set(held))
    to = dict(zip(source, target))
    tables = [[to.get(p, p) if x < h else p for x, p in enumerate(row)] for row, h in zip(a["tables"], a["held"])]
    shares = [0] * n_pages
    for p in held:
        shares[to.get(p, p)] = a["shares"][p]
    free = st["free"].cpu().tolist()
    free[:n_pages - u] = range(n_pages - 1, u - 1, -1)
    pad = [-1] * (n_pages // 2 - len(source))
    res = dict(tables_out=tables, shares_out=shares, free=free, n_free=[n_pages - u], source=source + pad,
               target=target + pad, count=[len(source)])
    k, v = st["k_cache"].clone(), st["v_cache"].clone()
    for s, t in to.items():
        k[:, t] = st["k_cache"][:, s]
        v[:, t] = st["v_cache"][:, s]
    return {**{x: _i32(y) for x, y in res.items()}, "k_cache": k, "v_cache": v}


def _exact_logprobs(st):
    res = {x: st[x].clone() if st[x].dtype == torch.int32 else st[x].double() for x in _logprobs_out(st)}
    k = st["case"]["top"]
    for i, t in enumerate(st["tokens"].tolist()):
        if t < 0:
            continue
        logp = torch.log_softmax(st["logits"][i].double(), -1)
        res["logprob"][i] = logp[t]
        res["entropy"][i] = -torch.special.xlogy(logp.exp(), logp.exp()).sum()
        order = torch.sort(st["logits"][i], descending=True, stable=True).indices
        res["rank"][i] = torch.nonzero(order == t)[0, 0]
        res["top_ids"][i] = order[:k]
        res["top_logprobs"][i] = logp[order[:k]]
    return res


_EXACT = {"chunk": _exact_chunk, "branch": _exact_branch, "compact": _exact_compact, "logprobs": _exact_logprobs}


def exact(case, seed):
    if case["op"] == "chunk" and work(case)["flops"] > 2.0e12:
        return None
    return _EXACT[case["op"]](prepare(case, seed))
