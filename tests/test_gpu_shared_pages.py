"""GPU parity of the operators of pages that several requests hold (page_fork,
page_free, page_compact, page_copy) against the oracle: whole numbers and
copies, equal."""

import random

import pytest
import torch

from oracle import paged as op
from test_gpu_paged import BF, F4, FH, i32, make_cache, pkg  # noqa: F401

pytestmark = pytest.mark.gpu


class State:
    """Tables, counts and stack on the host, the oracle's side."""

    def __init__(self, seed, B, W, page, lens, spare):
        r = random.Random(seed)
        self.page, self.lens = page, list(lens)
        self.held = [-(-n // page) for n in lens]
        self.P = sum(self.held) + spare
        pages = list(range(self.P))
        r.shuffle(pages)
        self.tables = [[-1 - r.randrange(3)] * W for _ in range(B)]
        for b in range(B):
            for j in range(self.held[b]):
                self.tables[b][j] = pages.pop()
        self.shares = [0] * self.P
        self.n_free = len(pages)
        self.free = pages + [-7] * (self.P - len(pages))

    def device(self):
        return dict(tables=i32(self.tables), held=i32(self.held), shares=i32(self.shares), free=i32(self.free),
                    n_free=i32([self.n_free]))

    def same(self, d):
        for name in ("tables", "held", "shares", "free"):
            assert d[name].tolist() == getattr(self, name), name
        assert d["n_free"].tolist() == [self.n_free]

    def fork(self, pkg, d, src, dst):
        ref = op.page_fork(src, dst, self.lens, self.tables, self.held, self.shares, self.free, self.n_free, self.page)
        got = pkg.page_fork(i32(src), i32(dst), i32(self.lens), d["tables"], d["held"], d["shares"], d["free"],
                            d["n_free"], self.page)
        for name in ("source", "target", "slots", "status"):
            assert getattr(got, name).tolist() == ref[name], name
        for name in ("tables", "held", "shares", "n_free"):
            setattr(self, name, ref[name])
        for s, t, st in zip(src, dst, ref["status"]):
            if st == 0:
                self.lens[t] = self.lens[s]
        self.same(d)
        return got

    def end(self, pkg, d, requests, keep=None):
        ref = op.page_free(requests, keep, self.tables, self.held, self.shares, self.free, self.n_free, self.page)
        got = pkg.page_free(i32(requests), d["tables"], d["held"], d["shares"], d["free"], d["n_free"], self.page,
                            keep=None if keep is None else i32(keep))
        assert got.tolist() == ref["status"]
        for name in ("held", "shares", "free", "n_free"):
            setattr(self, name, ref[name])
        for i, (r, st) in enumerate(zip(requests, ref["status"])):
            if st == 0:
                self.lens[r] = 0 if keep is None else keep[i]
        self.same(d)
        return ref["status"]

    def check_invariants(self):
        count = [0] * self.P
        for t, h in zip(self.tables, self.held):
            for p in t[:h]:
                count[p] += 1
        assert [max(c - 1, 0) for c in count] == self.shares
        assert sorted(self.free[:self.n_free]) == [p for p in range(self.P) if count[p] == 0]


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("seed", range(5))
def test_steps_of_forks_ends_and_growth(pkg, page, seed):
    r = random.Random(100 * page + seed)
    B, W = r.randint(2, 40), r.randint(2, 30)
    lens = [r.randint(0, W * page) if r.random() < 0.6 else 0 for _ in range(B)]
    s = State(seed, B, W, page, lens, r.choice([3, 40, 200]))
    d = s.device()
    for _ in range(8):
        src = [r.randrange(-1, B + 1) for _ in range(r.randint(1, B))]
        dst = [r.randrange(-1, B + 1) if r.random() < 0.3 else r.choice([b for b in range(B) if s.held[b] == 0] or [0])
               for _ in src]
        s.fork(pkg, d, src, dst)
        s.check_invariants()
        # Requests grow by the plan: every one by a few tokens, as far as pages go.
        lens = [min(W * page, n + r.randint(0, 20)) if s.held[b] else 0 for b, n in enumerate(s.lens)]
        plan = op.page_plan(lens, [0] * (B + 1), s.tables, s.held, s.free, s.n_free, page, 0)
        pkg.page_plan(i32(lens), i32([0] * (B + 1)), d["tables"], d["held"], d["free"], d["n_free"], page, n_rows=0)
        s.lens = [a if st == 0 else min(b, h * page) for a, b, h, st in zip(lens, s.lens, plan["held"], plan["status"])]
        for name in ("tables", "held", "free", "n_free"):
            setattr(s, name, plan[name])
        s.same(d)
        requests = [r.randrange(-1, B + 1) for _ in range(r.randint(1, B))]
        keep = None if r.random() < 0.3 else [r.choice([-1, 0, r.randint(0, W * page + 1),
                                                        max(0, s.lens[q % B] - r.randint(0, 5))]) for q in requests]
        s.end(pkg, d, requests, keep)
        s.check_invariants()


@pytest.mark.parametrize("B,W,page", [(600, 90, 16), (3000, 7, 64), (8192, 2, 16), (3, 20000, 16)])
def test_large_batches(pkg, B, W, page):
    r = random.Random(B)
    lens = [r.randint(0, W * page) if b < B // 3 else 0 for b in range(B)]
    s = State(B, B, W, page, lens, 2 * B)
    d = s.device()
    dst = list(range(B // 3, B))
    r.shuffle(dst)
    s.fork(pkg, d, [r.randrange(B // 3) if B > 3 else 0 for _ in dst], dst)
    s.check_invariants()
    ended = list(range(B))
    r.shuffle(ended)
    s.end(pkg, d, ended[:B // 2], [r.choice([0, s.lens[q]]) for q in ended[:B // 2]])
    s.check_invariants()
    s.end(pkg, d, list(range(B)))
    assert s.n_free == s.P and not any(s.shares) and not any(s.held)


def test_not_enough_pages(pkg):
    s = State(1, 8, 4, 16, [20, 16, 33, 0, 0, 0, 0, 0], 2)
    d = s.device()
    got = s.fork(pkg, d, [0, 1, 2, 0, 1], [3, 4, 5, 6, 7])
    assert got.status.tolist() == [0, 0, 0, 1, 0]          # whole pages are shared without a page of one's own
    s.check_invariants()


def test_refused_forks_and_ends(pkg):
    s = State(2, 6, 4, 16, [20, 40, 0, 0, 0, 64], 9)
    s.lens[5] = 65                                         # more than it holds
    d = s.device()
    got = s.fork(pkg, d, [0, 0, 0, 0, 6, -1, 5, 1, 2], [0, 1, 2, 2, 3, 3, 3, 4, 2])
    assert got.status.tolist() == [2, 2, 0, 2, 2, 2, 2, 0, 2]
    s.check_invariants()
    st = s.end(pkg, d, [0, 0, 1, 4, 6, -1, 2], [33, 0, 20, 31, 0, 0, -1])
    assert st == [2, 2, 2, 2, 2, 2, 2]      # more than held; named before; inside a shared page (both); not there; negative
    st = s.end(pkg, d, [4, 0], [16, 20])
    assert st == [0, 0]
    st = s.end(pkg, d, [1], [5])            # page 0 is still shared
    assert st == [2]
    st = s.end(pkg, d, [4])
    st = s.end(pkg, d, [1], [5])
    assert st == [0]
    s.check_invariants()


def test_entries_that_are_no_pages(pkg):
    s = State(3, 4, 4, 16, [64, 40, 0, 0], 5)
    s.tables[0][1], s.tables[0][2] = -3, 10 ** 6
    d = s.device()
    s.fork(pkg, d, [0, 1], [2, 3])
    s.end(pkg, d, [0, 2])


def test_nothing_to_do(pkg):
    s = State(4, 3, 2, 16, [5, 0, 0], 2)
    d = s.device()
    assert s.fork(pkg, d, [], []).status.numel() == 0
    s.end(pkg, d, [])
    s.fork(pkg, d, [1], [2])                               # of nothing
    s.end(pkg, d, [1, 2])


# ------------------------------------------------------------------ compact and copy
def compact(pkg, s, d, apart):
    ref = op.page_compact(s.tables, s.held, s.shares)
    kw = {}
    if apart:
        kw = dict(tables_out=torch.full_like(d["tables"], 99), shares_out=torch.full_like(d["shares"], 99))
    kept = {x: d[x].clone() for x in ("tables", "shares")}
    for _ in range(2 if apart else 1):
        got = pkg.page_compact(d["tables"], d["held"], d["shares"], d["free"], d["n_free"], **kw)
    assert got.tables.tolist() == ref["tables"] and got.shares.tolist() == ref["shares"]
    m = len(ref["source"])
    assert got.count.tolist() == [m] and d["n_free"].tolist() == [ref["n_free"]]
    assert got.source.tolist() == ref["source"] + [-1] * (s.P // 2 - m)
    assert got.target.tolist() == ref["target"] + [-1] * (s.P // 2 - m)
    assert d["free"].tolist()[:ref["n_free"]] == ref["free"]
    if apart:
        assert all(torch.equal(d[x], kept[x]) for x in kept)
    else:
        assert got.tables is d["tables"] and got.shares is d["shares"]
    return got


@pytest.mark.parametrize("apart", [True, False])
@pytest.mark.parametrize("B,W,page,spare", [(1, 1, 16, 0), (1, 3, 16, 1), (5, 9, 64, 30), (40, 50, 16, 0), (40, 50, 16, 700),
                                            (3, 3000, 32, 5000), (2000, 5, 16, 20000)])
def test_compact(pkg, B, W, page, spare, apart):
    r = random.Random(B + W)
    lens = [r.randint(0, W * page) if b % 3 < 2 else 0 for b in range(B)]
    s = State(B, B, W, page, lens, spare)
    d = s.device()
    empty = [b for b in range(B) if s.held[b] == 0]
    if empty:
        s.fork(pkg, d, [r.randrange(B) for _ in empty], empty)
    compact(pkg, s, d, apart)


def test_compact_without_held_pages_and_full(pkg):
    s = State(5, 3, 4, 16, [0, 0, 0], 50)
    compact(pkg, s, s.device(), True)
    s = State(6, 3, 4, 16, [64, 64, 64], 0)
    got = compact(pkg, s, s.device(), False)
    assert got.count.item() == 0


def test_compact_of_the_most_pages(pkg):
    P = 2 ** 20
    g = torch.Generator().manual_seed(1)
    pages = torch.randperm(P, generator=g)[:40000].int()
    tables = pages.view(4, 10000).cuda()
    held, shares = i32([10000, 9999, 0, 1]), torch.zeros(P, dtype=torch.int32, device="cuda")
    live = torch.cat([pages[:10000], pages[10000:19999], pages[30000:30001]]).sort().values
    free, n_free = torch.zeros(P, dtype=torch.int32, device="cuda"), i32([0])
    got = pkg.page_compact(tables, held, shares, free, n_free)
    u = live.numel()
    low = torch.zeros(u, dtype=torch.bool)
    low[live[live < u].long()] = True
    assert got.source[:int(got.count)].cpu().tolist() == live[live >= u].tolist()
    assert got.target[:int(got.count)].cpu().tolist() == torch.nonzero(~low)[:, 0].tolist()
    assert n_free.item() == P - u and free[:P - u].cpu().tolist() == list(range(P - 1, u - 1, -1))
    now = torch.cat([tables[0], tables[1][:9999], tables[3][:1]]).sort().values
    assert now.tolist() == list(range(u))


@pytest.mark.parametrize("dtype", [BF, FH])
@pytest.mark.parametrize("hd,nkv,page,layers,layout", [
    (64, 2, 64, 1, "pages"), (128, 4, 16, 3, "layers"), (128, 1, 256, 2, "pool"), (64, 3, 32, 2, "within"),
    (64, 3, 32, 0, "nhd"), (128, 2, 128, 0, "padded")])
@pytest.mark.parametrize("some", [False, True])
@pytest.mark.parametrize("n", [1, 9, 60])
def test_copy(pkg, dtype, hd, nkv, page, layers, layout, some, n):
    r = random.Random(n + page)
    P = 150
    if layout in ("nhd", "padded"):          # one layer, without its dimension
        k, v = make_cache(P, nkv, page, hd, dtype, layout)
    elif layout == "pool":
        k, v = torch.empty((layers, P, 2, nkv, page, hd), dtype=dtype, device="cuda").unbind(2)
    elif layout == "within":                 # the layers of a page side by side
        k, v = (torch.empty((P, layers, nkv, page, hd), dtype=dtype, device="cuda").transpose(0, 1) for _ in range(2))
    else:
        k, v = (torch.empty((layers, P, nkv, page, hd), dtype=dtype, device="cuda") for _ in range(2))
    for c in (k, v):
        c.copy_(torch.randn(c.shape, device="cuda"))
    pages = r.sample(range(P), 2 * n)
    source, target = pages[:n], pages[n:]
    source = [r.choice(source) for _ in source]             # a page may be copied many times
    slots = [r.choice([0, 1, r.randint(0, page), page, page + 3, -2]) for _ in source] if some else None
    count = r.randint(0, n + 2) if some else None
    if n > 5:
        source[1], target[2], source[3] = -1, P, 2 ** 31 - 1
    want = [k.clone(), v.clone()]
    for i in range(n if count is None else min(n, count)):
        if 0 <= source[i] < P and 0 <= target[i] < P:
            m = page if slots is None else min(max(slots[i], 0), page)
            for c in want:
                c[..., target[i], :, :m, :] = c[..., source[i], :, :m, :]
    pkg.page_copy(i32(source), i32(target), k, v, slots=None if slots is None else i32(slots),
                  count=None if count is None else i32([count]))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_copy_refusals(pkg):
    k, v = (torch.zeros((2, 9, 2, 16, 64), dtype=BF, device="cuda") for _ in range(2))
    s, t = i32([0]), i32([1])
    for a in ((k, k), (k[:1].expand(2, 9, 2, 16, 64), v), (k, v.transpose(0, 1))):
        with pytest.raises((pkg.SFError, ValueError)):
            pkg.page_copy(s, t, *a)
    for kw in (dict(slots=i32([1, 2])), dict(count=i32([])), dict(slots=t.long())):
        with pytest.raises(ValueError):
            pkg.page_copy(s, t, k, v, **kw)
    with pytest.raises(ValueError):
        pkg.page_copy(s, i32([1, 2]), k, v)
    with pytest.raises(ValueError):
        pkg.page_copy(s, t, k, v[:1])
    with pytest.raises((pkg.SFError, ValueError)):
        pkg.page_copy(s, t, k.float(), v.float())
    pkg.page_copy(s[:0], t[:0], k, v)


def test_arguments_refused(pkg):
    s = State(7, 3, 2, 16, [5, 0, 0], 2)
    d = s.device()
    a = (d["tables"], d["held"], d["shares"], d["free"], d["n_free"])
    for bad in ((i32([0]).long(), *a, 16), (i32([0]), d["tables"][:, :1], *a[1:], 16), (i32([0]), *a[:1], a[1][:2], *a[2:], 16)):
        with pytest.raises(ValueError):
            pkg.page_free(*bad)
    with pytest.raises(pkg.SFError):
        pkg.page_free(i32([0]), *a, 24)
    with pytest.raises(ValueError):
        pkg.page_fork(i32([0]), i32([1, 2]), i32(s.lens), *a, 16)
    with pytest.raises(pkg.SFError):
        pkg.page_fork(i32([0]), i32([1]), i32(s.lens), *a, 8)
    with pytest.raises(pkg.SFError):
        pkg.page_compact(*a[:3], d["free"][:2], d["n_free"])
    with pytest.raises(ValueError):
        pkg.page_compact(*a, tables_out=d["tables"][:2])
    s.same(d)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dt,hd", [(BF, 128), (FH, 64)])
def test_a_prompt_forked_continued_scored_and_packed(pkg, dt, hd):
    """A prompt run in chunks, forked into continuations that each append and
    attend, scored, the losers ended, the cache packed: at every step the
    attention is that of a cache that holds each request by itself."""
    B, W, page, nq, nkv, layers = 5, 12, 32, 6, 2, 2
    P = 40
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *shape: torch.randn(shape, dtype=dt, device="cuda", generator=g)
    k_cache, v_cache = (torch.zeros((layers, P, nkv, page, hd), dtype=dt, device="cuda") for _ in range(2))
    tables, held, shares = torch.zeros((B, W), dtype=torch.int32, device="cuda"), i32([0] * B), i32([0] * P)
    free, n_free = torch.randperm(P, device="cuda", generator=g).int(), i32([P])
    lens = [0] * B
    text = [[([], []) for _ in range(layers)] for _ in range(B)]      # every request's own keys and values

    def step(rows, chunk):
        """rows[b] new tokens of each request, appended and attended in every layer."""
        starts = [sum(rows[:b]) for b in range(B + 1)]
        for b in range(B):
            lens[b] += rows[b]
        n = starts[-1]
        plan = pkg.page_plan(i32(lens), i32(starts), tables, held, free, n_free, page, n_rows=n)
        assert plan.status.tolist() == [0] * B
        outs = []
        for layer in range(layers):
            q, k, v = rnd(n, nq, hd), rnd(n, nkv, hd), rnd(n, nkv, hd)
            pkg.kv_append(k, v, plan.slots, k_cache[layer], v_cache[layer])
            if chunk:
                out = pkg.chunk_attention(q, k_cache[layer], v_cache[layer], tables, i32(lens), starts=i32(starts),
                                          max_rows=max(rows))
            else:
                out = pkg.paged_attention(q, k_cache[layer], v_cache[layer], tables, i32(lens), starts=i32(starts),
                                          max_rows=max(rows))
            for b in range(B):
                text[b][layer][0].append(k[starts[b]:starts[b + 1]])
                text[b][layer][1].append(v[starts[b]:starts[b + 1]])
            outs.append((q, out))
        for layer, (q, out) in enumerate(outs):
            for b in range(B):
                if not rows[b]:
                    continue
                kk, vv = (torch.cat(x).double().transpose(0, 1).repeat_interleave(nq // nkv, 0) for x in text[b][layer])
                s, e = starts[b], starts[b + 1]
                x = q[s:e].double().transpose(0, 1) @ kk.transpose(1, 2) / hd ** 0.5
                pos = torch.arange(lens[b] - rows[b], lens[b], device="cuda")[:, None]
                x = x.masked_fill(torch.arange(lens[b], device="cuda")[None] > pos, float("-inf"))
                p = torch.softmax(x, -1)
                want, a = (p @ vv).transpose(0, 1), (p @ vv.abs()).transpose(0, 1)
                u = 2.0 ** -8 if dt == BF else 2.0 ** -11
                bound = (u + 2.0 ** -12) * a + (u + 2.0 ** -12) * want.abs() + 2.0 ** -25
                assert bool(((out[s:e].double() - want).abs() <= bound).all())

    step([130, 0, 0, 0, 0], True)
    step([85, 0, 0, 0, 0], True)
    copies = pkg.page_fork(i32([0, 0, 0]), i32([1, 2, 4]), i32(lens), tables, held, shares, free, n_free, page)
    assert copies.status.tolist() == [0, 0, 0] and copies.slots.tolist() == [215 % page] * 3
    pkg.page_copy(copies.source, copies.target, k_cache, v_cache, slots=copies.slots)
    for b in (1, 2, 4):
        lens[b] = lens[0]
        for layer in range(layers):
            for x in range(2):
                text[b][layer][x].extend(text[0][layer][x])
    for _ in range(3):
        step([1, 1, 1, 0, 1], False)
    scores = pkg.token_logprobs(torch.randn((4, 1000), device="cuda", generator=g), i32([5, 6, 7, 8]), top=3)
    order = scores.logprob.argsort().tolist()
    worst = [[0, 1, 2, 4][i] for i in order[:2]]
    assert pkg.page_free(i32(worst), tables, held, shares, free, n_free, page).tolist() == [0, 0]
    for b in worst:
        lens[b] = 0
        for layer in range(layers):
            text[b][layer][0].clear(), text[b][layer][1].clear()
    moves = pkg.page_compact(tables, held, shares, free, n_free)
    pkg.page_copy(moves.source, moves.target, k_cache, v_cache, count=moves.count)
    used = sum(h for b, h in enumerate(held.tolist())) - int(shares.sum())
    assert n_free.item() == P - used and int(max(tables[b][:h].max() for b, h in enumerate(held.tolist()) if h)) == used - 1
    rows = [0 if b in worst or lens[b] == 0 else 40 for b in range(B)]
    rows[3] = 90
    step(rows, True)
    step([1 if lens[b] else 0 for b in range(B)], False)
    everyone = [b for b in range(B) if lens[b]]
    pkg.page_free(i32(everyone), tables, held, shares, free, n_free, page)
    assert n_free.item() == P and not shares.any() and sorted(free.tolist()) == list(range(P))


def test_calls_on_another_stream_and_captured(pkg):
    s = State(8, 4, 6, 16, [90, 40, 0, 0], 9)
    d = s.device()
    src, dst, lens = i32([0, 1]), i32([2, 3]), i32(s.lens)
    k, v = (torch.randn((2, s.P, 2, 16, 64), device="cuda").to(BF) for _ in range(2))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    a = (d["tables"], d["held"], d["shares"], d["free"], d["n_free"])
    pkg.page_free(dst, *a, 16, stream=st)
    f = pkg.page_fork(src, dst, lens, *a, 16, stream=st)
    pkg.page_copy(f.source, f.target, k, v, slots=f.slots, stream=st)
    st.synchronize()
    ref = op.page_fork([0, 1], [2, 3], s.lens, s.tables, s.held, s.shares, s.free, s.n_free, 16)
    assert d["tables"].tolist() == ref["tables"] and d["shares"].tolist() == ref["shares"]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):     # the branches end and are forked again
        pkg.page_free(dst.flip(0), *a, 16)
        pkg.page_fork(src, dst, lens, *a, 16, *f)
        pkg.page_copy(f.source, f.target, k, v, slots=f.slots)
    for _ in range(3):
        graph.replay()
        assert d["tables"].tolist() == ref["tables"] and d["shares"].tolist() == ref["shares"]
        assert d["n_free"].tolist() == [ref["n_free"]]
        for i in range(2):
            m = int(f.slots[i])
            for c in (k, v):
                assert torch.equal(c[:, f.target[i], :, :m], c[:, f.source[i], :, :m])
