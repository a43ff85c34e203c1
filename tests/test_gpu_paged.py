"""GPU parity of the paged-cache operators against the float64 oracle.

page_plan is integers: equal. kv_append rounds fp32 arithmetic once to the
cache's type, so an element is off by at most half a step of that type plus
the fp32 rotation's three roundings.

paged_attention: with x the scaled scores, p the probabilities and A = sum p|v|
(the oracle's), an output is off by at most
  * the probabilities' rounding to the cache's type, u * A (u = half a step,
    2^-8 bf16, 2^-11 fp16; fp32 queries carry them exactly), and the output's
    own, u_out * |out|;
  * a relative error of every probability from its score: fp32 sums of hd
    products (each step may truncate: 2^-23 of the sum of magnitudes, qk), two
    roundings of the score and the exponential's 2^-22, which reach numerator
    and denominator; and the running sums, which add a piece for every 8 slots
    at least, each to 2^-23 of the sum: eps = 2 (hd + 8) 2^-23 max(qk, 1) +
    n / 8 * 2^-23 for n slots (2^-18 at least, for the rescalings and the join)
    times A and |out|.
The logarithm lse is off by eps.
"""

import ctypes
import math
import random

import pytest
import torch

from oracle import paged as op

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
BF, FH, F4 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__ as g
    g.build()
    import greedy_speculative_decoding_gb300 as p
    return p


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ page_plan
def plan_case(seed, B, W, page, tight=False, prompts=False, bad=False):
    r = random.Random(seed)
    held = [0 if prompts else r.randint(0, W) for _ in range(B)]
    lens = [r.choice([0, 1, r.randint(0, W * page), min(W * page, max(0, h * page + r.randint(-20, 20)))]) for h in held]
    rows = [n if prompts else min(n, r.randint(0, 5)) for n in lens]
    if bad:
        for b in r.sample(range(B), max(1, B // 4)):
            k = r.randint(0, 2)
            if k == 0:
                lens[b] = -r.randint(1, 2 ** 31 - 1)
            elif k == 1:
                lens[b] = W * page + r.randint(1, 2 ** 30)
            else:
                rows[b] = max(lens[b], 0) + 1
    need = [max(0, -(-n // page)) for n in lens]
    grow = sum(max(0, min(n, W) - h) for n, h in zip(need, held))
    spare = grow // 2 if tight else grow + 3
    cap = sum(held) + spare + 2
    pages = list(range(cap))
    r.shuffle(pages)
    tables, at = [[-1] * W for _ in range(B)], 0
    for b in range(B):
        tables[b][:held[b]] = pages[at:at + held[b]]
        at += held[b]
    free = pages[at:at + spare] + [-1] * (cap - spare)
    starts = [0]
    for n in rows:
        starts.append(starts[-1] + n)
    return lens, starts, tables, held, free, spare, page, starts[-1] + 3


def check_plan(pkg, case, in_place=False, repeat=1):
    lens, starts, tables, held, free, n_free, page, n_rows = case
    ref = op.page_plan(*case)
    t, h, f, nf = i32(tables), i32(held), i32(free), i32([n_free])
    for _ in range(repeat):
        kw = {} if in_place else dict(held_out=torch.full_like(h, -7), n_free_out=torch.full_like(nf, -7))
        res = pkg.page_plan(i32(lens), i32(starts), t, h, f, nf, page, n_rows=n_rows, **kw)
        got = dict(tables=t, held=res.held, free=f, n_free=res.n_free, status=res.status, slots=res.slots,
                   positions=res.positions)
        for name, x in got.items():
            want = [ref[name]] if name == "n_free" else ref[name]
            assert x.tolist() == want, name
    if in_place:
        assert res.held is h and res.n_free is nf
    else:
        assert h.tolist() == held and nf.tolist() == [n_free]


@pytest.mark.parametrize("B,W,page", [(1, 1, 16), (2, 9, 256), (8, 130, 64), (31, 5, 32), (32, 7, 16), (33, 64, 128),
                                      (1023, 6, 16), (1025, 3, 64), (8192, 2, 16)])
@pytest.mark.parametrize("tight", [False, True])
def test_plan(pkg, B, W, page, tight):
    check_plan(pkg, plan_case(B + W, B, W, page, tight))


@pytest.mark.parametrize("seed", range(8))
def test_plan_in_place_and_repeated(pkg, seed):
    r = random.Random(seed)
    case = plan_case(seed, r.randint(1, 60), r.randint(1, 40), r.choice([16, 32, 64, 128, 256]), seed % 2 == 1)
    check_plan(pkg, case, in_place=True)
    check_plan(pkg, case, repeat=3)


@pytest.mark.parametrize("B,W,page,tight", [(150, 120, 16, True), (9, 1500, 32, False), (1, 300, 16, False), (5, 700, 16, True), (200, 30, 64, True), (9, 1, 256, False)])
def test_plan_of_whole_prompts(pkg, B, W, page, tight):
    check_plan(pkg, plan_case(7 * B, B, W, page, tight, prompts=True))


@pytest.mark.parametrize("seed", range(4))
def test_plan_refuses_bad_requests_alone(pkg, seed):
    check_plan(pkg, plan_case(seed, 40, 11, 32, seed % 2 == 1, bad=True))


def test_plan_without_rows(pkg):
    lens, starts, tables, held, free, n_free, page, _ = plan_case(3, 12, 8, 16)
    check_plan(pkg, (lens, [0] * 13, tables, held, free, n_free, page, 0))
    check_plan(pkg, (lens, [4] * 13, tables, held, free, n_free, page, 9))


# ------------------------------------------------------------------ kv_append
def make_cache(n_pages, nkv, page, hd, dtype, layout="pages", fill=0.25):
    if layout == "pool":      # a page's keys and values side by side
        pool = torch.full((n_pages, 2, nkv, page, hd), fill, dtype=dtype, device="cuda")
        return pool[:, 0], pool[:, 1]
    if layout == "nhd":       # [page][head][dim] within a page
        k, v = (torch.full((n_pages, page, nkv, hd), fill, dtype=dtype, device="cuda") for _ in range(2))
        return k.transpose(1, 2), v.transpose(1, 2)
    if layout == "padded":    # rows of a slot, heads and pages apart
        k, v = (torch.full((n_pages, nkv + 1, page + 3, hd + 16), fill, dtype=dtype, device="cuda") for _ in range(2))
        return k[:, :nkv, :page, :hd], v[:, 1:, 3:, 16:]
    return tuple(torch.full((n_pages, nkv, page, hd), fill, dtype=dtype, device="cuda") for _ in range(2))


@pytest.mark.parametrize("din,dc", [(F4, BF), (F4, FH), (BF, BF), (FH, FH)])
@pytest.mark.parametrize("hd,nq,nkv,page,layout", [(64, 14, 2, 64, "pages"), (128, 4, 1, 16, "nhd"), (128, 5, 5, 256, "pool"),
                                                   (64, 3, 1, 32, "padded")])
@pytest.mark.parametrize("rope,fused,with_q", [(True, True, True), (True, False, False), (False, True, True)])
def test_append(pkg, din, dc, hd, nq, nkv, page, layout, rope, fused, with_q):
    g = torch.Generator(device="cuda").manual_seed(hd + nq + page)
    n, n_pages, n_pos = 37, 9, 50
    if fused:
        buf = torch.randn((n, (nq + 2 * nkv) * hd), dtype=din, device="cuda", generator=g)
        q, k, v = (x.view(n, -1, hd) for x in buf.split([nq * hd, nkv * hd, nkv * hd], dim=1))
    else:
        q, k, v = (torch.randn((n, h, hd), dtype=din, device="cuda", generator=g) for h in (nq, nkv, nkv))
    r = random.Random(5)
    slots = r.sample(range(n_pages * page), n)
    slots[3], slots[7], slots[11] = -1, n_pages * page, -2 ** 31
    pos = [r.randrange(n_pos) for _ in range(n)]
    pos[5], pos[6] = -1, n_pos
    cs = pkg.rope_table(n_pos, hd, 1e4) if rope else None
    k_cache, v_cache = make_cache(n_pages, nkv, page, hd, dc, layout)
    for q_dt in ({dc, din} if with_q else {None}):
        k_cache.fill_(0.25)
        v_cache.fill_(0.25)
        q_out = None if q_dt is None else torch.full((n, nq, hd), 0.5, dtype=q_dt, device="cuda")
        res = pkg.kv_append(k, v, i32(slots), k_cache, v_cache, q=q if with_q else None, q_out=q_out,
                            positions=i32(pos) if rope else None, rope=cs)
        assert res is q_out
        live = [i for i in range(n) if 0 <= slots[i] < n_pages * page and (not rope or 0 <= pos[i] < n_pos)]
        want = {}
        for name, src, turn in (("q", q, rope), ("k", k, rope), ("v", v, False)):
            x = src.cpu().double()
            y = x.clone()
            if turn:
                t = cs.cpu()
                for i in live:
                    for h in range(x.shape[1]):
                        y[i, h] = op.rotate(x[i, h], t[pos[i]])
            want[name] = (y, x.abs() + x.roll(hd // 2, -1).abs() if turn else torch.zeros_like(x))
        for name, got, fill, dt in (("q", q_out, 0.5, q_dt), ("k", k_cache, 0.25, dc), ("v", v_cache, 0.25, dc)):
            if got is None:
                continue
            y, mag = want[name]
            if name == "q":
                ref, m = torch.full_like(y, fill), torch.zeros_like(y)
                ref[live], m[live] = y[live], mag[live]
                out = got.cpu().double()
            else:
                ref = torch.full((n_pages * page, nkv, hd), fill, dtype=torch.float64)
                m = torch.zeros_like(ref)
                for i in live:
                    ref[slots[i]], m[slots[i]] = y[i], mag[i]
                out = got.transpose(1, 2).reshape(n_pages * page, nkv, hd).cpu().double()
            assert bool(((out - ref).abs() <= U[dt] * ref.abs() + 4 * 2.0 ** -24 * m + TINY[dt]).all()), name


def test_append_queries_in_place_and_one_row(pkg):
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((1, h, 64), dtype=BF, device="cuda", generator=g) for h in (4, 2, 2))
    cs = pkg.rope_table(1000, 64, 1e6)
    a, b = make_cache(2, 2, 16, 64, BF), make_cache(2, 2, 16, 64, BF)
    apart = pkg.kv_append(k, v, i32([17]), *a, q=q, positions=i32([999]), rope=cs)
    kept = q.clone()
    assert pkg.kv_append(k, v, i32([17]), *b, q=q, q_out=q, positions=i32([999]), rope=cs) is q
    assert torch.equal(q, apart) and not torch.equal(q, kept)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rope_table_is_the_engines_formula(pkg):
    t = pkg.rope_table(5000, 128, 1e6).double().cpu()
    i = torch.arange(64, dtype=torch.float64)
    ang = torch.arange(5000, dtype=torch.float64)[:, None] * torch.tensor(1e6, dtype=torch.float64) ** (-2 * i / 128)
    assert float((t - torch.stack([ang.cos(), ang.sin()], -1)).abs().max()) <= 2.0 ** -24 + 1e-11


# ------------------------------------------------------------------ attention
def attn_case(seed, lens, rows, nq, nkv, hd, page, dq=BF, dc=BF, layout="pages", tree=False, pad=2, q_scale=2.0,
              stale=None, strided_q=False):
    """Inputs of one call; cache slots that no request reaches hold `stale`."""
    r = random.Random(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(lens)
    held = [-(-n // page) for n in lens]
    W = max(1, max(held))
    n_pages = sum(held) + 2
    pages = list(range(n_pages))
    r.shuffle(pages)
    k, v = make_cache(n_pages, nkv, page, hd, dc, layout, float("nan") if stale is None else stale)
    tables, at = [[0] * W for _ in range(B)], 0
    for b in range(B):
        tables[b][:held[b]] = pages[at:at + held[b]]
        at += held[b]
        for i in range(held[b]):
            m = min(page, lens[b] - i * page)
            for c in (k, v):
                c[tables[b][i], :, :m] = torch.randn((nkv, m, hd), dtype=dc, device="cuda", generator=g)
    starts = [0]
    for x in rows:
        starts.append(starts[-1] + x)
    n = starts[-1] + pad
    if strided_q:
        q = (torch.randn((n, nq + 3, hd + 16), dtype=dq, device="cuda", generator=g) * q_scale)[:, 2:2 + nq, 8:8 + hd]
    else:
        q = torch.randn((n, nq, hd), dtype=dq, device="cuda", generator=g) * q_scale
    mask = None
    if tree:
        mask = [0] * n
        for b in range(B):
            for j in range(rows[b]):
                m = 1 << j
                if j:
                    m |= mask[starts[b] + r.randrange(j)]
                mask[starts[b] + j] = m if r.random() < 0.9 else 0
        mask = [m - (1 << 64) if m >> 63 else m for m in mask]
    return dict(q=q, k=k, v=v, tables=tables, lens=lens, starts=starts, mask=mask, max_rows=max(1, max(rows)))


def call(pkg, c, **kw):
    out = torch.full(c["q"].shape, 7.0, dtype=c["q"].dtype, device="cuda")
    lse = torch.full(c["q"].shape[:2], 7.0, device="cuda")
    mask = None if c["mask"] is None else torch.tensor(c["mask"], dtype=torch.int64, device="cuda")
    a = dict(starts=i32(c["starts"]), max_rows=c["max_rows"], mask=mask, out=out, lse=lse)
    a.update(kw)
    res = pkg.paged_attention(c["q"], c["k"], c["v"], i32(c["tables"]), i32(c["lens"]), **a)
    assert a["out"] is None or res is a["out"]
    return res, a["lse"]


def check_attn(c, out, lse, scale=None):
    hd = c["q"].shape[2]
    scale = 1 / math.sqrt(hd) if scale is None else scale
    ref, rl, A, qk, live = op.paged_attention(c["q"].cpu(), c["k"].cpu(), c["v"].cpu(), c["tables"], c["lens"],
                                              c["starts"], scale, c["mask"], c["max_rows"])
    out, lse = out.double().cpu(), lse.double().cpu()
    assert bool((out[~live] == 7).all() and (lse[~live] == 7).all())
    up = 0.0 if c["q"].dtype == F4 else U[c["k"].dtype]
    slots = min(max(c["lens"]), len(c["tables"][0]) * c["k"].shape[2])
    eps = 2 * (hd + 8) * 2.0 ** -23 * qk.clamp(min=1.0) + max(2.0 ** -18, slots / 8 * 2.0 ** -23)
    bound = (up + eps[..., None]) * A + (U[c["q"].dtype] + eps[..., None]) * ref.abs() + TINY[c["q"].dtype]
    err = (out - ref).abs()
    assert bool((err[live] <= bound[live]).all()), float((err / bound)[live].max())
    empty = rl == float("-inf")
    assert bool((lse[live] == rl[live])[empty[live]].all())
    assert bool(((lse - rl).abs() <= eps)[live & ~empty.all(1)][~empty[live & ~empty.all(1)]].all())


LENS = [[1], [0, 1, 15, 16, 17], [63, 64, 65, 0, 0], [128, 200, 1, 511], [1000]]


@pytest.mark.parametrize("dq,dc", [(BF, BF), (FH, FH), (F4, BF)])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("lens", LENS)
def test_one_token(pkg, dq, dc, hd, lens):
    """Single new tokens: group 7, page 16; empty requests among them."""
    c = attn_case(hd + len(lens), lens, [min(1, n) for n in lens], 14, 2, hd, 16, dq, dc)
    check_attn(c, *call(pkg, c))


@pytest.mark.parametrize("nq,nkv", [(1, 1), (8, 1), (4, 4), (10, 2), (16, 1), (17, 1), (40, 8), (66, 2)])
@pytest.mark.parametrize("rows", [1, 3, 9])
def test_head_layouts(pkg, nq, nkv, rows):
    c = attn_case(nq + rows, [77, 9, 130], [rows] * 3, nq, nkv, 64, 32)
    check_attn(c, *call(pkg, c))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["pages", "pool", "nhd", "padded"])
@pytest.mark.parametrize("hd", [64, 128])
def test_pages_and_cache_layouts(pkg, page, layout, hd):
    c = attn_case(page, [page - 1, page, page + 1, 3 * page + 5], [1, 2, 3, 4], 4, 2, hd, page, layout=layout,
                  strided_q=True)
    check_attn(c, *call(pkg, c))


@pytest.mark.parametrize("dq,dc", [(BF, BF), (FH, FH), (F4, BF)])
@pytest.mark.parametrize("rows", [2, 5, 9, 16, 17, 33, 64])
def test_tree_masks(pkg, dq, dc, rows):
    """Masked rows, some of which see nothing of the pass; requests that are
    nothing but the pass's rows leave such rows empty."""
    c = attn_case(rows, [rows, rows + 1, 100 + rows, rows], [rows, rows, rows, 1], 6, 2, 64, 16, dq, dc, tree=True)
    check_attn(c, *call(pkg, c))


@pytest.mark.parametrize("dq,dc", [(BF, BF), (F4, BF)])
@pytest.mark.parametrize("rows", [1, 7, 40, 80])
def test_many_rows(pkg, dq, dc, rows):
    c = attn_case(rows, [rows, 300 + rows, rows + 63], [rows, rows, max(1, rows - 1)], 14, 2, 128, 64, dq, dc)
    check_attn(c, *call(pkg, c))


def test_ragged_rows_and_requests_without_rows(pkg):
    c = attn_case(5, [70, 33, 0, 129, 5, 64], [3, 0, 0, 9, 5, 1], 4, 2, 128, 32, pad=4)
    check_attn(c, *call(pkg, c))


def test_rows_past_max_rows_and_past_n_are_left(pkg):
    c = attn_case(6, [50, 60], [6, 6], 4, 2, 64, 16, pad=0)
    c["max_rows"] = 4
    check_attn(c, *call(pkg, c))
    c = attn_case(6, [50, 60], [6, 6], 4, 2, 64, 16, pad=0)
    out, lse = call(pkg, c)
    # The same call told of fewer rows than starts promises writes those alone.
    short = dict(c, q=c["q"][:9])
    o9, l9 = call(pkg, short)
    assert torch.equal(o9, out[:9]) and torch.equal(l9, lse[:9])


def test_more_rows_than_tokens(pkg):
    """Rows before position 0 see nothing."""
    c = attn_case(8, [3, 40], [3, 2], 4, 2, 64, 16)
    c["starts"] = [0, 5, 7]
    c["q"] = torch.randn(9, 4, 64, device="cuda").to(BF)
    c["max_rows"] = 5
    check_attn(c, *call(pkg, c))


def test_without_starts(pkg):
    c = attn_case(9, [30, 70, 12], [2, 2, 2], 4, 2, 64, 16, pad=0)
    a, la = call(pkg, c)
    b, lb = call(pkg, c, starts=None, max_rows=None)
    assert torch.equal(a, b) and torch.equal(la, lb)
    check_attn(c, a, la)


def test_scale_and_no_lse(pkg):
    for scale in (1.0, -0.3, 0.0):
        c = attn_case(10, [90, 33], [1, 4], 4, 2, 64, 16, q_scale=1.0)
        out, lse = call(pkg, c, scale=scale)
        check_attn(c, out, lse, scale)
        o2, _ = call(pkg, c, scale=scale, lse=None)
        assert torch.equal(out[:5], o2[:5])


def test_lens_past_the_table_and_pages_outside_the_cache(pkg):
    c = attn_case(11, [64, 100], [1, 2], 4, 2, 64, 16, stale=0.5)
    c["lens"] = [10 ** 9, 100]      # cut to the table's width
    c["tables"][0] = [c["tables"][0][i % 4] for i in range(len(c["tables"][0]))]
    c["tables"][1][2], c["tables"][1][5] = -5, c["k"].shape[0]   # read as zeros
    check_attn(c, *call(pkg, c))
    c["lens"] = [-3, 100]           # nothing to see
    check_attn(c, *call(pkg, c))


@pytest.mark.parametrize("dq,dc", [(BF, BF), (FH, FH), (F4, BF)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("tree", [False, True])
def test_masked_nan_and_inf_change_nothing(pkg, dq, dc, bad, tree):
    """Keys and values of later rows, other branches and slots past the
    length: whatever they hold, rows that do not see them stay the same."""
    rows = 9
    c = attn_case(12, [100, rows, 64 + 3], [rows, rows, 6], 14, 2, 64, 16, dq, dc, tree=tree, stale=bad)
    good, lgood = call(pkg, c)
    check_attn(c, good, lgood)
    # Spoil the last row's slot of every request: only rows that see it change.
    spoiled = []
    for b, n in enumerate(c["lens"]):
        pg, off = c["tables"][b][(n - 1) // 16], (n - 1) % 16
        c["k"][pg, 0, off] = bad
        c["v"][pg, :, off] = bad
        r = c["starts"][b + 1] - c["starts"][b]
        for j in range(r):
            m = c["mask"][c["starts"][b] + j] if tree else (1 << (j + 1)) - 1
            if (m >> (r - 1)) & 1:
                spoiled.append(c["starts"][b] + j)
    out, lse = call(pkg, c)
    keep = [i for i in range(good.shape[0]) if i not in spoiled]
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], lgood[keep])
    assert spoiled and not bool(torch.isfinite(out[spoiled][:, 7:]).any())   # head 1: V alone is spoiled


@pytest.mark.parametrize("dq,hd,nq,nkv,rows,lens", [
    (BF, 128, 10, 2, 9, [20011, 64, 9000]), (FH, 64, 14, 2, 13, [9000, 30000]), (BF, 64, 16, 2, 16, [40000]),
    (BF, 128, 8, 2, 1, [33000, 1, 700]), (F4, 128, 14, 2, 9, [7000]), (BF, 128, 12, 4, 11, [300] * 40)])
@pytest.mark.parametrize("tree", [False, True])
def test_long_contexts(pkg, dq, hd, nq, nkv, rows, lens, tree):
    """Many units a CTA, items shared by many CTAs, several items a CTA."""
    c = attn_case(rows + hd, lens, [min(n, rows) for n in lens], nq, nkv, hd, 64, dq, BF if dq == F4 else dq, tree=tree)
    check_attn(c, *call(pkg, c))


@pytest.mark.parametrize("dq", [BF, F4])
@pytest.mark.parametrize("rows", [1, 5, 9])
@pytest.mark.parametrize("down", [False, True])
def test_maxima_that_grow_along_the_cache(pkg, dq, rows, down):
    """Keys grow (or shrink) with the slot, so that the running maximum rises
    by many powers of two from unit to unit."""
    n = 2000
    c = attn_case(31, [n, 130], [rows, rows], 14, 2, 64, 32, dq, BF, q_scale=1.0)
    f = torch.logspace(2, -2, n, base=10.0) if down else torch.logspace(-2, 2, n, base=10.0)
    for s in range(n):
        c["k"][c["tables"][0][s // 32], :, s % 32] *= float(f[s])
    check_attn(c, *call(pkg, c))


def test_large_scores(pkg):
    """Scores far apart and far from zero: the running maximum is followed."""
    c = attn_case(13, [500, 3], [2, 3], 4, 2, 64, 16, q_scale=60.0)
    check_attn(c, *call(pkg, c))


def test_same_result_in_every_run_and_on_another_stream(pkg):
    c = attn_case(14, [700, 33, 64, 1300], [9, 2, 9, 1], 14, 2, 128, 32)
    a, la = call(pkg, c)
    s = torch.cuda.Stream()
    for _ in range(3):
        s.wait_stream(torch.cuda.current_stream())
        b, lb = call(pkg, c, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_two_calls_at_once(pkg):
    """Two streams, a workspace each (allocated by the calls)."""
    cs = [attn_case(15 + i, [900 + i, 40], [3, 1], 14, 2, 128, 32) for i in range(2)]
    want = [call(pkg, c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = []
    for _ in range(5):
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append(call(pkg, c))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


def test_captured_pass_replayed_with_other_lengths(pkg):
    """Plan, append and attention captured once; replays read new lengths."""
    nq, nkv, hd, page, B, R, W = 4, 2, 64, 16, 3, 2, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = make_cache(30, nkv, page, hd, BF, fill=0.0)
    lens, starts = i32([0] * B), i32([0, R, 2 * R, 3 * R])
    tables, held, free, n_free = i32([[0] * W] * B), i32([0] * B), i32(list(range(30))), i32([30])
    q, k, v = (torch.zeros((B * R, h, hd), dtype=BF, device="cuda") for h in (nq, nkv, nkv))
    cs = pkg.rope_table(W * page, hd, 1e4)
    out, lse = torch.zeros_like(q), torch.zeros((B * R, nq), device="cuda")
    ws = pkg.paged_attention_workspace(q, kc, tables, R)
    plan = pkg.PagePlan(i32([0] * B * R), i32([0] * B * R), held, n_free, i32([0] * B))

    def one_pass():
        pkg.page_plan(lens, starts, tables, held, free, n_free, page, slots=plan.slots, positions=plan.positions,
                      status=plan.status)
        qr = pkg.kv_append(k, v, plan.slots, kc, vc, q=q, positions=plan.positions, rope=cs)
        pkg.paged_attention(qr, kc, vc, tables, lens, starts=starts, max_rows=R, out=out, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lens.fill_(R)
        one_pass()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one_pass()
    hist = [[] for _ in range(B)]      # (k, v) of every committed token, as the cache holds them
    now = [0] * B
    r = random.Random(4)
    lens.fill_(0)
    for step in range(40):
        for x, h in ((q, nq), (k, nkv), (v, nkv)):
            x.copy_(torch.randn((B * R, h, hd), device="cuda", generator=g))
        now = [x + R if x + R <= W * page else R for x in now]
        lens.copy_(i32(now))
        graph.replay()
        torch.cuda.synchronize()
        assert plan.status.tolist() == [0] * B
        assert sorted(free.tolist()[:n_free.item()] + [p for b in range(B) for p in tables[b].tolist()[:held[b].item()]]) \
            == list(range(30))
        cq = torch.zeros_like(q)
        for b in range(B):
            hist[b] = hist[b][:now[b] - R]
            for j in range(R):
                i, pos = b * R + j, now[b] - R + j
                rot = [op.rotate(k[i, h].cpu(), cs[pos].cpu()).to(BF) for h in range(nkv)]
                hist[b].append((torch.stack(rot), v[i].cpu()))
                for h in range(nq):
                    cq[i, h] = op.rotate(q[i, h].cpu(), cs[pos].cpu()).to(BF)
        for b in range(B):
            kk = torch.stack([x[0] for x in hist[b]]).double()
            vv = torch.stack([x[1] for x in hist[b]]).double()
            for j in range(R):
                seen = torch.zeros(now[b], dtype=torch.bool)
                seen[:now[b] - R + j + 1] = True
                for h in range(nq):
                    ref, _, A, qk = op.attention(cq[b * R + j, h].cpu(), kk[:, h // 2], vv[:, h // 2], 0.125, seen)
                    # Beside the operator's own bound: the oracle's rotated rows may round to
                    # the other bf16 neighbour (an error of 2^-7 of a key or query), which
                    # moves a score by at most 2 * 2^-7 * qk.
                    eps = 2 * 2.0 ** -6 * max(qk, 1.0)
                    err = (out[b * R + j, h].double().cpu() - ref).abs()
                    assert bool((err <= (2.0 ** -8 + eps) * A + (2.0 ** -8 + eps) * ref.abs() + 1e-30).all())
        # Some guesses are rejected: the next pass starts from fewer tokens.
        now = [max(0, x - r.randint(0, R)) if r.random() < 0.9 else 0 for x in now]


def test_offsets_past_32_bits(pkg):
    """Pages whose keys lie more than 2^31 elements into the cache."""
    nkv, page, hd = 8, 256, 128
    per = nkv * page * hd
    n_pages = (2 ** 31 + 2 ** 27) // per
    k = torch.zeros((n_pages, nkv, page, hd), dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = [n_pages - 1, 0, n_pages - 3, n_pages - 2]
    kr, vr = (torch.randn((700, nkv, hd), dtype=BF, device="cuda", generator=g) for _ in range(2))
    slots = [ids[s // page] * page + s % page for s in range(700)]
    pkg.kv_append(kr, vr, i32(slots), k, v)
    small_k, small_v = k[torch.tensor(ids, device="cuda")], v[torch.tensor(ids, device="cuda")]
    assert torch.equal(small_k.transpose(1, 2).reshape(-1, nkv, hd)[:700], kr)
    q = torch.randn((2, 16, hd), dtype=BF, device="cuda", generator=g)
    c = dict(q=q, k=k, v=v, tables=[ids], lens=[700], starts=[0, 2], mask=None, max_rows=2)
    out, lse = call(pkg, c)
    c.update(k=small_k, v=small_v, tables=[[0, 1, 2, 3]])
    o2, l2 = call(pkg, c)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    check_attn(c, out, lse)


def test_many_requests(pkg):
    r = random.Random(1)
    lens = [r.choice([0, 1, r.randint(1, 60)]) for _ in range(1500)]
    c = attn_case(21, lens, [min(1, n) for n in lens], 2, 1, 64, 16)
    check_attn(c, *call(pkg, c))


def test_wrapper_refusals(pkg):
    c = attn_case(22, [30], [1], 4, 2, 64, 16)
    for kw in (dict(max_rows=None), dict(workspace=torch.empty(1, dtype=torch.uint8, device="cuda")),
               dict(lse=torch.empty(2, 3, device="cuda")), dict(out=torch.empty(3, 4, 32, dtype=BF, device="cuda")),
               dict(starts=i32([0, 1, 2])), dict(mask=i32([1, 2, 3])), dict(mask=torch.ones(3, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call(pkg, c, **kw)
    with pytest.raises(ValueError):
        pkg.kv_append(c["k"][:, 0], c["v"][:, 0], i32([0]), c["k"], c["v"])
    with pytest.raises(ValueError):
        pkg.page_plan(i32([1]), i32([0, 1]), i32([[0]]), i32([0]), i32([0]), i32([1]), 16)
    with pytest.raises(pkg.SFError):
        pkg.page_plan(i32([1]), i32([0, 1]), i32([[0]]), i32([0]), i32([0]), i32([1]), 17, n_rows=1)


# ------------------------------------------- the larger tiles, on small inputs
# A table wide enough for long requests: the query tile is chosen from what the
# tables can hold, so these run in tiles of 32 (17 to 32 queries a KV head) and
# of 128 queries, as long caches do.
def wide(c):
    c["tables"] = [t + [-1] * (70000 // c["k"].shape[2]) for t in c["tables"]]
    return c


TILES = [(3, 14, 2), (9, 14, 2), (40, 8, 2), (64, 5, 1), (30, 14, 2)]   # 21, 63, 160, 320, 210 queries
TYPES = [(BF, BF), (FH, FH), (F4, BF)]


@pytest.mark.parametrize("dq,dc", TYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows,nq,nkv", TILES)
@pytest.mark.parametrize("tree", [False, True])
def test_large_tiles(pkg, dq, dc, hd, rows, nq, nkv, tree):
    """Requests that are nothing but the pass's rows (with a mask, rows that
    see nothing among them), empty ones, ones that end at a unit's border."""
    lens = [rows, 300 + rows, 0, rows + 1, 128, 192 + rows, 64]
    c = wide(attn_case(rows + hd, lens, [min(rows, n) if n != 128 else 1 for n in lens], nq, nkv, hd, 32, dq, dc, tree=tree))
    check_attn(c, *call(pkg, c))


@pytest.mark.parametrize("dq,dc", TYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [3, 9])
@pytest.mark.parametrize("down", [False, True])
def test_large_tiles_with_growing_maxima(pkg, dq, dc, hd, rows, down):
    n = 1500
    c = wide(attn_case(37, [n, 130], [rows, rows], 14, 2, hd, 32, dq, dc, q_scale=1.0))
    f = torch.logspace(2, -2, n, base=10.0) if down else torch.logspace(-2, 2, n, base=10.0)
    for s in range(n):
        c["k"][c["tables"][0][s // 32], :, s % 32] *= float(f[s])
    check_attn(c, *call(pkg, c))


@pytest.mark.parametrize("dq,dc", TYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [3, 9])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_large_tiles_with_masked_nan_and_inf(pkg, dq, dc, hd, rows, tree, bad):
    """As test_masked_nan_and_inf_change_nothing."""
    c = wide(attn_case(14, [200, rows, 64 + 3], [rows, rows, min(rows, 6)], 14, 2, hd, 16, dq, dc, tree=tree, stale=bad))
    good, lgood = call(pkg, c)
    check_attn(c, good, lgood)
    spoiled = []
    for b, n in enumerate(c["lens"]):
        pg, off = c["tables"][b][(n - 1) // 16], (n - 1) % 16
        c["k"][pg, 0, off] = bad
        c["v"][pg, :, off] = bad
        r = c["starts"][b + 1] - c["starts"][b]
        for j in range(r):
            m = c["mask"][c["starts"][b] + j] if tree else (1 << (j + 1)) - 1
            if (m >> (r - 1)) & 1:
                spoiled.append(c["starts"][b] + j)
    out, lse = call(pkg, c)
    keep = [i for i in range(good.shape[0]) if i not in spoiled]
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], lgood[keep])
    assert spoiled and not bool(torch.isfinite(out[spoiled][:, 7:]).any())   # head 1: V alone is spoiled


@pytest.mark.parametrize("dq,dc", TYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [3, 9])
def test_large_tiles_of_strided_queries_and_other_scales(pkg, dq, dc, hd, rows):
    for scale in (1.0, -0.3, 0.0):
        c = wide(attn_case(41, [90, 333, 2], [1, rows, 2], 14, 2, hd, 64, dq, dc, q_scale=1.0, strided_q=True))
        check_attn(c, *call(pkg, c, scale=scale), scale)
        c["q"] = c["q"] * 40.0   # scores far apart
        check_attn(c, *call(pkg, c), None)
    c = wide(attn_case(43, [30, 70, 12], [rows] * 3, 14, 2, hd, 16, dq, dc, pad=0))
    c["max_rows"] = 2            # rows behind it are left as they were
    check_attn(c, *call(pkg, c))
    c["lens"] = [2, 70, -1]      # rows before position 0 see nothing
    check_attn(c, *call(pkg, c))


@pytest.mark.parametrize("hd,nq", [(64, 40), (128, 40), (128, 7)])
def test_fp32_sums_over_long_caches(pkg, hd, nq):
    """Sums over hundreds of units a CTA keep fp32 accuracy: the tensor cores
    cut off each product's addition, but no sum they keep is of more than 16
    units of 12 products, 2^-23 of it each. Beside that, the fp32 additions of
    those sums and of the parts (128 of 2^-24 at most), and the scores, small
    here (qk): 2 (2^-22 + (hd + 8) 2^-23 qk). The values are positive, so that
    the bound is relative to the output. The table repeats 40 pages, which
    leaves the softmax's mean as it is."""
    g = torch.Generator(device="cuda").manual_seed(hd + nq)
    page, cycle, times, B = 256, 40, 190, 2
    k = torch.randn((cycle, 1, page, hd), dtype=BF, device="cuda", generator=g)
    v = torch.randn((cycle, 1, page, hd), dtype=BF, device="cuda", generator=g).abs()
    q = torch.randn((B, nq, hd), device="cuda", generator=g) * 1e-3
    tables = i32([list(range(cycle)) * times] * B)
    out = pkg.paged_attention(q, k, v, tables, i32([page * cycle * times] * B)).double()
    kd, vd = k.double().reshape(-1, hd), v.double().reshape(-1, hd)
    ref = torch.softmax(q.double() @ kd.T / math.sqrt(hd), -1) @ vd
    qk = float((q.double().abs() @ kd.abs().T).max()) / math.sqrt(hd)
    bound = 192 * 2.0 ** -23 + 128 * 2.0 ** -24 + 2 * (2.0 ** -22 + (hd + 8) * 2.0 ** -23 * qk)
    assert float(((out - ref).abs() / ref).max()) <= bound


@pytest.mark.parametrize("B,rows", [(3, 2), (90, 1), (90, 5)])
def test_passes_back_to_back(pkg, B, rows):
    """Sixty passes enqueued without a pause (each kernel may come up while
    the one before it ends) leave what the same calls leave one at a time."""
    nq, nkv, hd, page, W, passes = 8, 2, 64, 16, 24, 60
    cap, n = B * W, B * rows
    g = torch.Generator(device="cuda").manual_seed(B + rows)
    r = random.Random(B)
    at, lens = [r.randint(0, 60) for _ in range(B)], []
    for p in range(passes):
        for b in range(B):   # some requests end and begin again
            at[b] = rows if r.random() < 0.05 or at[b] + rows > W * page else at[b] + rows
        lens.append(i32(at))
    starts = i32([b * rows for b in range(B + 1)])
    rope = pkg.rope_table(W * page, hd, 1e4)
    q, k, v = (torch.randn((passes, n, h, hd), dtype=BF, device="cuda", generator=g) for h in (nq, nkv, nkv))

    def run(pause):
        tables = torch.zeros((B, W), dtype=torch.int32, device="cuda")
        held, free, nf = i32([0] * B), torch.arange(cap, dtype=torch.int32, device="cuda"), i32([cap])
        kc = torch.zeros((cap, nkv, page, hd), dtype=BF, device="cuda")
        vc = torch.zeros_like(kc)
        slots, pos, status = i32([0] * n), i32([0] * n), i32([0] * B)
        qr = torch.zeros((n, nq, hd), dtype=BF, device="cuda")
        out = torch.zeros((passes, n, nq, hd), dtype=BF, device="cuda")
        ws = pkg.paged_attention_workspace(q[0], kc, tables, rows)
        steps = []
        for p in range(passes):
            steps.append(lambda p=p: pkg.page_plan(lens[p], starts, tables, held, free, nf, page, slots=slots, positions=pos,
                                                   status=status))
            steps.append(lambda p=p: pkg.kv_append(k[p], v[p], slots, kc, vc, q=q[p], q_out=qr, positions=pos, rope=rope))
            steps.append(lambda p=p: pkg.paged_attention(qr, kc, vc, tables, lens[p], starts=starts, max_rows=rows,
                                                         out=out[p], workspace=ws))
        torch.cuda.synchronize()
        for s in steps:
            s()
            if pause:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert int(status.abs().sum()) == 0
        return out, kc, vc, tables, held, nf

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


# One item (request and KV head) a CTA, in tiles of 16, 32 or 128 queries: as
# many requests as it takes, all over the same pages.
ITEMS = [(1, 7), (3, 7), (9, 7)]   # rows, query heads of a KV head


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows,group", ITEMS)
@pytest.mark.parametrize("gap", [12, 16, 18])
@pytest.mark.parametrize("at", [0, 40000])
def test_fp16_tail_behind_dominant_slots(pkg, hd, rows, group, gap, at):
    """Four slots (of one unit, apart) whose score lies `gap` above that of
    65536 others and whose values are 0: the output is the others' alone, each
    with a probability of e^-gap of the largest. Scores are exact here. Beside
    half a step of each probability and of the output, a probability in fp16
    may be off by 2^-37 of the largest (half its smallest step, 2^-25, as the
    probabilities are scaled by 2^12 at least). eps: rounding of the scaled
    score (|x| <= 2 gap log2 e: two roundings of 2^-24, to the base 2) and of
    the exponential (2^-22); the sums of probabilities and values lose at most
    2^-23 for every 16 slots."""
    nkv, page, n = 2, 256, 65536 + 256
    B = 160
    g = torch.Generator(device="cuda").manual_seed(gap)
    k = torch.zeros((n // page, nkv, page, hd), dtype=FH, device="cuda")
    v = torch.randn((n // page, nkv, page, hd), dtype=FH, device="cuda", generator=g).abs()
    for s in (0, 16, 32, 48):
        k[(at + s) // page, :, (at + s) % page, 0] = gap
        v[(at + s) // page, :, (at + s) % page] = 0
    q = torch.zeros((B * rows, nkv * group, hd), dtype=FH, device="cuda")
    q[:, :, 0] = 1.0
    width = 140000 // page   # (wide enough for tiles of 128)
    tables = torch.arange(width, dtype=torch.int32, device="cuda").clamp(max=n // page - 1).repeat(B, 1)
    lse = torch.zeros((B * rows, nkv * group), device="cuda")
    out = pkg.paged_attention(q, k, v, tables, i32([n] * B), max_rows=rows, scale=1.0, lse=lse).double()
    w = torch.full((n,), math.exp(-gap), dtype=torch.float64, device="cuda")
    w[at:at + 64:16] = 1.0
    vd = v.transpose(0, 1).reshape(nkv, n, hd).double()
    eps = 2 * (4 * gap * 1.4427 * 2.0 ** -24 + 2.0 ** -22) + n / 16 * 2.0 ** -23
    for j in range(rows):
        m = n - rows + j + 1
        total = w[:m].sum()
        ref = ((w[:m, None] * vd[:, :m]).sum(1) / total).repeat_interleave(group, 0)        # [heads, hd]
        bound = 2 * (U[FH] + eps) * ref + m * 2.0 ** -37 * float(vd.max()) / total + TINY[FH]
        err = (out[j::rows] - ref).abs()
        assert bool((err <= bound).all()), float((err / bound).max())
        assert float((lse[j::rows].double() - gap - torch.log(total)).abs().max()) <= eps


@pytest.mark.parametrize("dt", [BF, FH])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows,group", ITEMS)
def test_16_bit_sums_over_long_items(pkg, dt, hd, rows, group):
    """Items of 2^20 slots, one a CTA. The tensor cores cut off what they add,
    always to the same side, so no sum that they keep is of more than 256 units
    of four products, 2^-23 of it each; the additions of those sums are 64 of
    2^-24. Keys are 0 (every probability exactly the largest, sums of them
    exact) and values positive; the output's own rounding, half a step at most
    for each element, averages out over the outputs that differ (five standard
    deviations of a uniform error)."""
    nkv, page, cycle, B = 8, 256, 16, 40
    g = torch.Generator(device="cuda").manual_seed(hd)
    k = torch.zeros((cycle, nkv, page, hd), dtype=dt, device="cuda")
    v = torch.randn((cycle, nkv, page, hd), dtype=dt, device="cuda", generator=g).abs() + 0.5
    q = torch.ones((B * rows, nkv * group, hd), dtype=dt, device="cuda")
    W = 2 ** 20 // page
    tables = (torch.arange(W, dtype=torch.int32, device="cuda") % cycle).repeat(B, 1)
    lse = torch.zeros((B * rows, nkv * group), device="cuda")
    out = pkg.paged_attention(q, k, v, tables, i32([2 ** 20] * B), max_rows=rows, lse=lse).double()
    ends = v[-1].double().flip(1).cumsum(1)                    # sums of the last slots
    mean = []
    for j in range(rows):                                      # row j does not see the last rows - 1 - j
        x = v.double().sum((0, 2)) * (W // cycle) - (ends[:, rows - 2 - j] if j < rows - 1 else 0)
        mean.append((x / (2 ** 20 - (rows - 1 - j))).repeat_interleave(group, 0))
    ref = torch.stack(mean).repeat(B, 1, 1)
    rel = out / ref - 1
    sums = 1024 * 2.0 ** -23 + 64 * 2.0 ** -24
    assert float(rel.abs().max()) <= U[dt] + sums
    assert abs(float(rel.mean())) <= sums + 5 * U[dt] / math.sqrt(3 * nkv * hd)
    seen = torch.tensor([2 ** 20 - (rows - 1 - j) for j in range(rows)], dtype=torch.float64, device="cuda").log()
    assert float((lse.double() - seen.repeat(B)[:, None]).abs().max()) <= 2.0 ** -17


@pytest.mark.parametrize("dq,dc", TYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows,group", ITEMS)
def test_sums_of_like_probabilities(pkg, dq, dc, hd, rows, group):
    """Items of 2^20 slots, one a CTA, nearly all with one probability that is
    no power of two: fp32 sums of them err the same way at every step, half a
    step (2^-24) at most. No sum is of more than 1024 + 16 + 32 steps (fp32
    queries in tiles of 128: 32 within a unit, 16 units, 1024 times those;
    others have 128 or 256 units and 128 or 64 times those). Beside that the
    exponential (2^-22), the rounding of the scaled score (two of 2^-24, times
    log2 e * 1.25) and of the logarithm (2^-24 * 16, twice)."""
    nkv, page, cycle, B = 8, 256, 16, 40
    g = torch.Generator(device="cuda").manual_seed(hd)
    k = torch.zeros((cycle, nkv, page, hd), dtype=dc, device="cuda")
    k[:, :, 1:, 0] = -1.2
    q = torch.zeros((B * rows, nkv * group, hd), dtype=dq, device="cuda")
    q[:, :, 0] = 1.0
    W = 2 ** 20 // page
    tables = (torch.arange(W, dtype=torch.int32, device="cuda") % cycle).repeat(B, 1)
    lse = torch.zeros((B * rows, nkv * group), device="cuda")
    v = torch.randn((cycle, nkv, page, hd), dtype=dc, device="cuda", generator=g)
    pkg.paged_attention(q, k, v, tables, i32([2 ** 20] * B), max_rows=rows, scale=1.0, lse=lse)
    p = math.exp(float(k[0, 0, 1, 0]))
    want = torch.tensor([math.log(W + (W * 255 - (rows - 1 - j)) * p) for j in range(rows)], dtype=torch.float64)
    bound = 1072 * 2.0 ** -24 + 2.0 ** -22 + 4 * 2.0 ** -24 + 32 * 2.0 ** -24
    assert float((lse.double().cpu() - want.repeat(B)[:, None]).abs().max()) <= bound


def test_plan_of_the_most_rows(pkg):
    """2^31 - 1 rows, the last 300 those of one request: nothing is written
    behind them, where the last four indexes end at 2^31."""
    n = 2 ** 31 - 1
    slots, pos = (torch.full((n + 5,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    tables, held = torch.zeros((1, 8), dtype=torch.int32, device="cuda"), i32([0])
    res = pkg.page_plan(i32([500]), i32([n - 300, n]), tables, held, torch.arange(40, dtype=torch.int32, device="cuda"),
                        i32([40]), 64, slots=slots[:n], positions=pos[:n])
    assert res.status.tolist() == [0] and tables.tolist() == [list(range(39, 31, -1))]
    p = torch.arange(200, 500)
    assert pos[n - 300:].tolist() == p.tolist() + [77] * 5
    assert slots[n - 300:].tolist() == ((39 - p // 64) * 64 + p % 64).tolist() + [77] * 5
    assert int(slots[:n - 300].max()) == -1 and int(slots[:n - 300].min()) == -1
    assert int(pos[:n - 300].max()) == 0 and int(pos[:n - 300].min()) == 0


def test_inputs_that_require_grad(pkg):
    """No gradient would come back: refused, unless gradients are off."""
    c = attn_case(51, [30, 9], [2, 1], 4, 2, 64, 16)
    ref, _ = call(pkg, c)
    for name in ("q", "k", "v"):
        d = dict(c)
        d[name] = c[name].clone().requires_grad_()
        with pytest.raises(ValueError, match="requires grad"):
            call(pkg, d)
        with torch.no_grad():
            assert torch.equal(call(pkg, d)[0], ref)
    k, v, q = (torch.zeros((3, h, 64), dtype=BF, device="cuda") for h in (2, 2, 4))
    rope, pos = pkg.rope_table(9, 64, 1e4), i32([0, 1, 2])
    for name in ("k", "v", "q", "rope", "q_out"):
        a = dict(k=k, v=v, q=q, rope=rope, q_out=torch.zeros_like(q))
        a[name] = a[name].clone().requires_grad_()
        with pytest.raises(ValueError, match="requires grad"):
            pkg.kv_append(a["k"], a["v"], i32([1, 2, -1]), c["k"], c["v"], q=a["q"], q_out=a["q_out"], positions=pos,
                          rope=a["rope"])


def test_tensors_written_in_place_are_marked_so(pkg):
    """What a call writes counts as changed in place, so that a graph which has
    saved it notices; with tensors of inference mode nothing is counted."""
    c = attn_case(52, [30, 9], [2, 1], 4, 2, 64, 16)
    tables, held, free, n_free = i32([[0] * 4] * 2), i32([0, 0]), i32(list(range(9))), i32([9])
    q, out, lse = c["q"], torch.zeros_like(c["q"]), torch.zeros(c["q"].shape[:2], device="cuda")
    x = torch.ones_like(c["k"], requires_grad=True)
    y = (x * c["k"]).sum()
    new = [tables, held, free, n_free, c["k"], c["v"], out, lse]
    before, kept = [t._version for t in new], q._version
    plan = pkg.page_plan(i32([30, 9]), i32(c["starts"]), tables, held, free, n_free, 16, n_rows=3)
    rows = torch.randn((3, 2, 64), device="cuda").to(BF)
    pkg.kv_append(rows, rows, i32([1, 2, 3]), c["k"], c["v"])
    call(pkg, c, out=out, lse=lse)
    assert all(t._version > b for t, b in zip(new, before)) and q._version == kept and plan.slots._version > 0
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        k, v = torch.zeros_like(c["k"]), torch.zeros_like(c["v"])
    pkg.kv_append(rows, rows, i32([1, 2, 3]), k, v)
    assert torch.equal(k[0, :, 1:4], rows.transpose(0, 1))


def terms(x, n):
    """x rounded to n bf16 terms (as fp32 queries and probabilities are held: n = 3)."""
    x, out = x.float(), torch.zeros_like(x.float())
    for _ in range(n):
        t = (x - out).bfloat16().float()
        out = out + t
    return out.double()


def third_term_case(hd, rows, prior):
    """fp32 queries over `prior` slots that all rows see (keys 0 but for slot 1),
    and nothing of the pass's own; tiles of 16, 32 (hd 64) or 128 queries."""
    nkv, group, page = 2, 7, 64
    pages = -(-(prior + rows) // page)
    k = torch.zeros((pages, nkv, page, hd), dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    tables = torch.zeros((1, 140000 // page), dtype=torch.int32, device="cuda")
    tables[0, :pages] = torch.arange(pages, dtype=torch.int32, device="cuda")
    mask = torch.zeros(rows, dtype=torch.int64, device="cuda")
    return k, v, tables, mask, nkv * group


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [1, 3, 9])
@pytest.mark.parametrize("prior", [2, 128])
def test_third_term_of_fp32_queries(pkg, hd, rows, prior):
    """Scores that are the third term alone: a query of 1 + 2^-9 + d and 1 +
    2^-9 (d below 2^-17) against a key of 1 and -1. The other two terms cancel,
    and the products of each term are one step of the tensor cores, which cut
    off at most 2^-23 of the magnitudes: 2 in the last step, 2^-8 before. The
    scale 2^17 makes that 2^-5 and the score d * 2^17 = 0.5 to 1."""
    k, v, tables, mask, nq = third_term_case(hd, rows, prior)
    k[0, :, 1, 0::2], k[0, :, 1, 1::2] = 1.0, -1.0
    q = torch.zeros((rows, nq, hd), device="cuda")
    d = torch.zeros((rows, nq), dtype=torch.float64)
    for j in range(rows):
        for h in range(nq):
            i = (j * nq + h) * 5 % (hd // 2) * 2          # a pair of dimensions
            big = 2.0 ** -18 + (1 + (j + 3 * h) % 15) * 2.0 ** -22
            d[j, h] = big
            a, b = (1 + 2.0 ** -9 + big, 1 + 2.0 ** -9) if h % 2 else (-(1 + 2.0 ** -9), -(1 + 2.0 ** -9 + big))
            q[j, h, i], q[j, h, i + 1] = a, b
    assert torch.equal(terms(q, 3), q.double()) and torch.equal(q[:, :, 0::2].sum(2) - q[:, :, 1::2].sum(2), d.float().cuda())
    lse = torch.zeros((rows, nq), device="cuda")
    pkg.paged_attention(q, k, v, tables, i32([prior + rows]), starts=i32([0, rows]), max_rows=rows, mask=mask,
                        scale=2.0 ** 17, lse=lse)
    s = d * 2.0 ** 17
    want = torch.log(torch.exp(s) + (prior - 1))
    bound = 1.01 * 2.0 ** -5 * torch.exp(s - want) * math.exp(2.0 ** -5) + 2.0 ** -20
    gone = (want - math.log(prior)).abs()                  # what the score is without the third term: 0
    assert bool((gone > 4 * bound).all())
    assert bool(((lse.double().cpu() - want).abs() <= bound).all())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [1, 3, 9])
@pytest.mark.parametrize("prior", [2, 128])
def test_third_term_of_fp32_probabilities(pkg, hd, rows, prior):
    """Outputs 1 - p, with p from 1/2 to 1 next to a slot of probability 1: p is
    off by 2^-22 of it from the exponential and 2^-23 from the scaled score (two
    roundings of 2^-24, times ln 2), the last step of the tensor cores by 2^-23 of
    a magnitude of 2, fp32 sums, the division and the output by 2^-23 together,
    relative to 1 and not to the difference: 2^-20 in all. The third term is up
    to 2^-18."""
    k, v, tables, mask, nq = third_term_case(hd, rows, prior)
    k[0, :, 1, 0] = -1.0
    v[0, :, 0], v[0, :, 1] = 1.0, -1.0
    q = torch.zeros((rows, nq, hd), device="cuda")
    q[:, :, 0] = 0.03 + 0.65 * torch.linspace(0, 1, rows * nq, dtype=torch.float64).view(rows, nq).float()
    out = torch.zeros_like(q)
    pkg.paged_attention(q, k, v, tables, i32([prior + rows]), starts=i32([0, rows]), max_rows=rows, mask=mask, scale=1.0,
                        out=out)
    p = torch.exp(-q[:, :, 0].double().cpu())
    total = prior - 1 + p
    assert float((terms(p, 2) - p).abs().max()) > 3 * 2.0 ** -20
    assert float((out.double().cpu() * total[..., None] - (1 - p)[..., None]).abs().max()) <= 2.0 ** -20


@pytest.mark.parametrize("dt", [BF, FH])
@pytest.mark.parametrize("R,group,cap", [(2, 2, 20), (9, 5, 20), (9, 5, 6)])
def test_captured_pass_step_by_step(pkg, dt, R, group, cap):
    """A captured plan, append and attention, replayed over requests that grow,
    give guesses back, finish and begin anew: after every replay the plan's
    numbers are the oracle's, every slot of the cache holds what was put there
    last to one rounding, and the attention is the oracle's over the cache and
    the rotated queries that are there."""
    nkv, hd, page, B, W = 2, 64, 16, 3, 8
    nq, n = nkv * group, 3 * R
    g = torch.Generator(device="cuda").manual_seed(8)
    r = random.Random(6)
    kc, vc = make_cache(cap, nkv, page, hd, dt, fill=0.0)
    lens, starts = i32([0] * B), i32([0, R, 2 * R, 3 * R])
    tables, held, free, n_free = i32([[0] * W] * B), i32([0] * B), i32(list(range(cap))), i32([cap])
    q, k, v = (torch.zeros((n, h, hd), dtype=dt, device="cuda") for h in (nq, nkv, nkv))
    cs = pkg.rope_table(W * page, hd, 1e4)
    qr, out, lse = torch.zeros_like(q), torch.zeros_like(q), torch.zeros((n, nq), device="cuda")
    ws = pkg.paged_attention_workspace(q, kc, tables, R)
    slots, pos, status = i32([0] * n), i32([0] * n), i32([0] * B)

    def one_pass():
        pkg.page_plan(lens, starts, tables, held, free, n_free, page, slots=slots, positions=pos, status=status)
        pkg.kv_append(k, v, slots, kc, vc, q=q, q_out=qr, positions=pos, rope=cs)
        pkg.paged_attention(qr, kc, vc, tables, lens, starts=starts, max_rows=R, out=out, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one_pass()                     # (more rows than tokens: every request is refused)
    torch.cuda.current_stream().wait_stream(side)
    assert status.tolist() == [2] * B
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one_pass()
    book = dict(tables=tables.tolist(), held=held.tolist(), free=free.tolist(), n_free=cap)
    want_k, want_v = (torch.zeros((cap * page, nkv, hd), dtype=torch.float64) for _ in range(2))
    mag = torch.zeros_like(want_k)
    now, short = [0] * B, 0
    t = cs.cpu()
    for step in range(25):
        for x, h in ((q, nq), (k, nkv), (v, nkv)):
            x.copy_(torch.randn((n, h, hd), device="cuda", generator=g))
        out.fill_(7.0)
        lse.fill_(7.0)
        now = [x + R if x + R <= W * page else R for x in now]
        lens.copy_(i32(now))
        graph.replay()
        torch.cuda.synchronize()
        ref = op.page_plan(now, starts.tolist(), book["tables"], book["held"], book["free"], book["n_free"], page, n)
        got = dict(tables=tables, held=held, free=free, status=status, slots=slots, positions=pos)
        for name, x in got.items():
            assert x.tolist() == ref[name], (step, name)
        assert n_free.tolist() == [ref["n_free"]]
        book = {x: ref[x] for x in ("tables", "held", "free", "n_free")}
        hk, hv, hq, hr = k.cpu(), v.cpu(), q.cpu(), qr.cpu().double()
        for i in range(n):
            s, p = ref["slots"][i], ref["positions"][i]
            if s < 0:
                continue
            for h in range(nkv):
                want_k[s, h], mag[s, h] = op.rotate(hk[i, h], t[p]), hk[i, h].abs() + hk[i, h].roll(hd // 2).abs()
                want_v[s, h] = hv[i, h].double()
            for h in range(nq):
                y = op.rotate(hq[i, h], t[p])
                m = (hq[i, h].abs() + hq[i, h].roll(hd // 2).abs()).double()
                assert bool(((hr[i, h] - y).abs() <= U[dt] * y.abs() + 4 * 2.0 ** -24 * m + TINY[dt]).all())
        flat_k, flat_v = (c.transpose(1, 2).reshape(-1, nkv, hd).cpu().double() for c in (kc, vc))
        assert bool(((flat_k - want_k).abs() <= U[dt] * want_k.abs() + 4 * 2.0 ** -24 * mag + TINY[dt]).all())
        assert torch.equal(flat_v, want_v)
        # (a request that got no pages keeps its table: its rows are not looked at)
        served = [x == 0 for x in ref["status"]]
        short += served.count(False)
        rows = torch.tensor([b * R + j for b in range(B) if served[b] for j in range(R)], dtype=torch.long)
        at, some = [b for b in range(B) if served[b]], [0]
        for _ in at:
            some.append(some[-1] + R)
        o, l = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
        o[:len(rows)], l[:len(rows)] = out[rows.cuda()], lse[rows.cuda()]
        if at:
            check_attn(dict(q=torch.cat([qr[rows.cuda()], qr[:n - len(rows)]]), k=kc, v=vc, starts=some, mask=None,
                            max_rows=R, tables=[book["tables"][b] for b in at], lens=[now[b] for b in at]), o, l)
        # Some guesses are rejected, some requests finish: the next pass starts from fewer tokens.
        now = [max(0, (x if s else x - R) - r.randint(0, R)) if r.random() < 0.9 else 0 for x, s in zip(now, served)]
    assert cap > 6 or short > 0


def test_every_call_on_a_stream_of_its_own(pkg):
    """A pass on a stream that is not the current one: the same as on the
    current one, what the calls allocate included."""
    B, R, nq, nkv, hd, page, W = 3, 2, 8, 2, 64, 16, 6
    g = torch.Generator(device="cuda").manual_seed(9)
    q, k, v = (torch.randn((B * R, h, hd), dtype=BF, device="cuda", generator=g) for h in (nq, nkv, nkv))
    lens, starts = i32([5, 40, 96]), i32([0, R, 2 * R, 3 * R])

    def one_pass(stream):
        tables, held, free, nf = torch.zeros((B, W), dtype=torch.int32, device="cuda"), i32([0] * B), i32(list(range(20))), i32([20])
        kc, vc = make_cache(20, nkv, page, hd, BF, fill=0.5)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        rope = pkg.rope_table(W * page, hd, 1e4, stream=stream)
        plan = pkg.page_plan(lens, starts, tables, held, free, nf, page, n_rows=B * R, stream=stream)
        qr = pkg.kv_append(k, v, plan.slots, kc, vc, q=q, positions=plan.positions, rope=rope, stream=stream)
        out = pkg.paged_attention(qr, kc, vc, tables, lens, starts=starts, max_rows=R, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        return [rope, *plan, tables, free, kc, vc, qr, out]

    want = one_pass(None)
    for a, b in zip(want, one_pass(torch.cuda.Stream())):
        assert torch.equal(a, b)


def test_calls_with_nothing_to_do(pkg):
    """No rows, no requests: nothing is written, nothing is refused."""
    c = attn_case(53, [30, 9], [2, 1], 4, 2, 64, 16)
    kept = c["k"].clone()
    none = torch.empty((0, 2, 64), dtype=BF, device="cuda")
    q0 = torch.empty((0, 4, 64), dtype=BF, device="cuda")
    rope = pkg.rope_table(4, 64, 1e4)
    assert pkg.kv_append(none, none, i32([]), c["k"], c["v"], q=q0, positions=i32([]), rope=rope).shape == (0, 4, 64)
    assert torch.equal(c["k"].nan_to_num(3.0), kept.nan_to_num(3.0))
    assert pkg.paged_attention(q0, c["k"], c["v"], i32(c["tables"]), i32([30, 9]), starts=i32([0, 0, 0]),
                               max_rows=1).shape == (0, 4, 64)
    out = torch.full_like(c["q"], 7.0)
    pkg.paged_attention(c["q"], c["k"], c["v"], torch.empty((0, 3), dtype=torch.int32, device="cuda"), i32([]), out=out)
    pkg.paged_attention(c["q"], c["k"], c["v"], i32(c["tables"]), i32([30, 9]), starts=i32([0, 0, 0]), max_rows=3, out=out)
    assert bool((out == 7).all())


@pytest.mark.parametrize("dq,dc", TYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows,group", [(3, 7), (9, 7), (9, 1)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("start", [16384, 16383, 16380])
def test_masked_nan_where_sums_move(pkg, dq, dc, hd, rows, group, bad, start):
    """Items of 257 units, one a CTA, whose last unit is where output and sums
    move to the part and holds the pass's own rows (for some starts the unit
    before it as well): values there that are no finite numbers reach no row
    that does not see them, and the rest is the mean it should be."""
    nkv, page, B, cycle = 2, 64, 160, 8
    n = start + rows
    g = torch.Generator(device="cuda").manual_seed(start + rows)
    k, v = (torch.randn((cycle + 2, nkv, page, hd), dtype=dc, device="cuda", generator=g) for _ in range(2))
    W = 140000 // page
    tables = (torch.arange(W, dtype=torch.int32, device="cuda") % cycle).repeat(B, 1)
    tables[:, start // page:start // page + 2] = torch.tensor([cycle, cycle + 1], dtype=torch.int32, device="cuda")
    q = torch.randn((rows, nkv * group, hd), device="cuda", generator=g).to(dq).repeat(B, 1, 1)
    lse = torch.zeros(q.shape[:2], device="cuda")
    good = pkg.paged_attention(q, k, v, tables, i32([n] * B), max_rows=rows, lse=lse)
    at = start + rows - 1                      # the last row's slot: only that row sees it
    k[cycle + at // page - start // page, :, at % page] = bad
    v[cycle + at // page - start // page, :, at % page] = bad
    l2 = torch.zeros_like(lse)
    out = pkg.paged_attention(q, k, v, tables, i32([n] * B), max_rows=rows, lse=l2)
    keep = torch.tensor([i for i in range(B * rows) if i % rows != rows - 1], device="cuda")
    assert torch.equal(out[keep], good[keep]) and torch.equal(l2[keep], lse[keep])
    assert not bool(torch.isfinite(out[rows - 1::rows]).any())
    ids = tables[0, :n // page + 1].long()
    kd, vd = (c[ids].transpose(0, 1).reshape(nkv, -1, hd).double() for c in (k, v))
    for j in range(rows - 1):
        x = torch.einsum("hgd,hsd->hgs", q[j].double().view(nkv, group, hd), kd[:, :start + j + 1]) / math.sqrt(hd)
        qk = torch.einsum("hgd,hsd->hgs", q[j].double().abs().view(nkv, group, hd), kd[:, :start + j + 1].abs()).amax(-1)
        p = torch.softmax(x, -1)
        ref, A = torch.einsum("hgs,hsd->hgd", p, vd[:, :start + j + 1]), torch.einsum("hgs,hsd->hgd", p, vd[:, :start + j + 1].abs())
        # (as check_attn; the sums over units: 512 of the tensor cores' steps and the folds)
        eps = 2 * (hd + 8) * 2.0 ** -23 * (qk / math.sqrt(hd)).clamp(min=1.0)[..., None] + 1100 * 2.0 ** -23
        up = 0.0 if dq == F4 else U[dc]
        bound = (up + eps) * A + (U[dq] + eps) * ref.abs() + TINY[dq]
        if dq == FH:
            bound = bound + n * 2.0 ** -37 * float(vd[:, :start + j + 1].abs().max()) * p.amax(-1)[..., None]
        err = (good[j::rows].double().view(B, nkv, group, hd) - ref).abs()
        assert bool((err <= bound).all()), float((err / bound).max())
