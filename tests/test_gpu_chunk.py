"""GPU parity of chunk_attention against the float64 oracle. Bounds as derived
for paged_attention (test_gpu_paged.py): probabilities and outputs rounded by
half a step of their type, and scores and sums in fp32.

Which kernel a call takes follows what its tables can hold, so small cases are
run twice: in tables that the requests fill (the kernels of few queries), and in
wide ones (the kernel of many, when there are more than 128 queries)."""

import math
import random

import pytest
import torch

from oracle import paged as op
from test_gpu_paged import BF, F4, FH, TINY, U, attn_case, i32, pkg  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = [(BF, BF), (FH, FH), (F4, BF)]


def widened(c, wide):
    """The tables, wide ones with entries behind the requests' pages that are no pages."""
    if not wide:
        return i32(c["tables"])
    more = max(0, 2 ** 17 // c["k"].shape[2] - len(c["tables"][0]))
    return torch.nn.functional.pad(i32(c["tables"]), (0, more), value=2 ** 30)


def call(pkg, c, wide=False, **kw):
    out = torch.full(c["q"].shape, 7.0, dtype=c["q"].dtype, device="cuda")
    lse = torch.full(c["q"].shape[:2], 7.0, device="cuda")
    a = dict(starts=i32(c["starts"]), max_rows=c["max_rows"], out=out, lse=lse)
    a.update(kw)
    res = pkg.chunk_attention(c["q"], c["k"], c["v"], widened(c, wide), i32(c["lens"]), **a)
    assert a["out"] is None or res is a["out"]
    return res, a["lse"]


def both(pkg, c, scale=None, rows=None, **kw):
    ref = reference(c, scale)
    for wide in (False, True):
        check(c, *call(pkg, c, wide, **({} if scale is None else dict(scale=scale)), **kw), scale, rows, ref)


def reference(c, scale=None):
    scale = 1 / math.sqrt(c["q"].shape[2]) if scale is None else scale
    return op.chunk_attention(c["q"].cpu(), c["k"].cpu(), c["v"].cpu(), c["tables"], c["lens"], c["starts"], scale)


def check(c, out, lse, scale=None, rows=None, ref=None):
    """rows: the rows compared (default all)."""
    hd = c["q"].shape[2]
    ref, rl, A, qk, live = ref or reference(c, scale)
    out, lse = out.double().cpu(), lse.double().cpu()
    assert bool((out[~live] == 7).all() and (lse[~live] == 7).all())
    up = 0.0 if c["q"].dtype == F4 else U[c["k"].dtype]
    slots = min(max(c["lens"]), len(c["tables"][0]) * c["k"].shape[2])
    eps = 2 * (hd + 8) * 2.0 ** -23 * qk.clamp(min=1.0) + max(2.0 ** -18, slots / 8 * 2.0 ** -23)
    bound = (up + eps[..., None]) * A + (U[c["q"].dtype] + eps[..., None]) * ref.abs() + TINY[c["q"].dtype]
    if rows is not None:
        live = live & rows
    err = (out - ref).abs()
    assert bool((err[live] <= bound[live]).all()), float((err / bound)[live].max())
    empty = rl == float("-inf")
    assert bool((lse == rl)[live][empty[live]].all())
    assert bool(((lse - rl).abs() <= eps)[live][~empty[live]].all())


# ------------------------------------------------------------------ sizes
@pytest.mark.parametrize("dq,dc", TYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("lens,rows", [([1], [1]), ([81], [81]), ([127, 128, 129], [127, 128, 129]),
                                       ([300, 0, 1, 255, 257], [300, 0, 1, 100, 2]), ([1100], [90]), ([700], [513])])
def test_sizes(pkg, dq, dc, hd, lens, rows):
    c = attn_case(len(lens) + lens[0], lens, rows, 4, 2, hd, 64, dq, dc)
    both(pkg, c)


@pytest.mark.parametrize("dq,dc", [(BF, BF), (F4, BF)])
@pytest.mark.parametrize("nq,nkv", [(1, 1), (3, 3), (8, 1), (14, 2), (10, 2), (28, 4), (66, 2), (130, 1)])
def test_head_layouts(pkg, dq, dc, nq, nkv):
    c = attn_case(nq, [150, 401], [150, 99], nq, nkv, 64, 32, dq, dc)
    both(pkg, c)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["pages", "pool", "nhd", "padded"])
@pytest.mark.parametrize("hd", [64, 128])
def test_pages_and_cache_layouts(pkg, page, layout, hd):
    c = attn_case(page + hd, [530, 97, 1029], [200, 97, 333], 6, 2, hd, page, BF, BF, layout)
    both(pkg, c)


@pytest.mark.parametrize("dq,dc", TYPES)
@pytest.mark.parametrize("hd,nq,nkv,lens,rows", [(128, 28, 4, [2100], [1037]), (128, 40, 8, [1500, 640], [129, 640]),
                                                 (64, 14, 2, [4099, 33, 2000], [450, 33, 1])])
def test_model_layouts(pkg, dq, dc, hd, nq, nkv, lens, rows):
    c = attn_case(nq, lens, rows, nq, nkv, hd, 64, dq, dc)
    both(pkg, c)


@pytest.mark.parametrize("dq", [BF, FH])
def test_many_ragged_requests(pkg, dq):
    r = random.Random(3)
    lens = [r.choice([0, r.randint(1, 60), r.randint(1, 700)]) for _ in range(70)]
    rows = [r.randint(0, n) for n in lens]
    rows[5], lens[5] = 333, 600
    c = attn_case(9, lens, rows, 4, 1, 64, 16, dq, dq)
    both(pkg, c)


# ------------------------------------------------------------------ rows and tables out of the ordinary
@pytest.mark.parametrize("dq,dc", TYPES)
def test_more_rows_than_tokens(pkg, dq, dc):
    """The first rows have negative positions: they see nothing."""
    c = attn_case(1, [300, 5, 0, 200], [300, 5, 0, 200], 4, 2, 128, 64, dq, dc)
    c["lens"] = [190, 0, 0, 1]
    for wide in (False, True):
        out, lse = call(pkg, c, wide)
        check(c, out, lse)
        assert bool((out[:110] == 0).all() and (lse[:110] == float("-inf")).all())


@pytest.mark.parametrize("dq", [BF, F4])
def test_without_starts(pkg, dq):
    c = attn_case(2, [300, 301, 400], [120, 120, 120], 4, 2, 64, 64, dq, BF, pad=0)
    both(pkg, c, starts=None, max_rows=None)
    out = pkg.chunk_attention(c["q"], c["k"], c["v"], i32(c["tables"]), i32(c["lens"]))
    check(c, out, call(pkg, c)[1])


def test_rows_past_max_rows_and_past_n_are_left(pkg):
    c = attn_case(4, [400, 300], [200, 150], 4, 2, 64, 64, pad=0)
    live = torch.ones(350, dtype=torch.bool)
    live[170:200] = False
    for wide in (False, True):
        out, lse = call(pkg, c, wide, max_rows=170)
        assert bool((out[170:200] == 7).all() and (lse[170:200] == 7).all())
        check(c, out, lse, rows=live)
        out, lse = call(pkg, c, wide, starts=i32([0, 200, 500]), max_rows=300)     # rows up to 500 of 350
        assert bool(torch.isfinite(out).all())


def test_lens_past_the_table_and_pages_outside_the_cache(pkg):
    c = attn_case(5, [500, 400], [130, 100], 4, 2, 64, 64)
    c["tables"][0][3], c["tables"][1][0] = -5, 10 ** 6                  # read as zeros
    both(pkg, c)
    for lens, rows in (([512], [130]), ([2 ** 17], [700])):             # (the second in wide tables)
        c = attn_case(6, lens, rows, 4, 2, 64, 64)
        c["lens"] = [lens[0] + 5000]
        check(c, *call(pkg, c))


@pytest.mark.parametrize("dq,dc", TYPES)
@pytest.mark.parametrize("scale", [0.0, -0.07, 1.3])
def test_scales_and_strided_queries(pkg, dq, dc, scale):
    c = attn_case(8, [333, 150], [222, 150], 6, 3, 128, 64, dq, dc, strided_q=True)
    for wide in (False, True):
        out, lse = call(pkg, c, wide, scale=scale)
        check(c, out, lse, scale=scale)
        buf = torch.full((c["q"].shape[0], 9, 160), 7.0, dtype=dq, device="cuda")
        strided, lse = call(pkg, c, wide, scale=scale, out=buf[:, 1:7, 16:144])
        assert torch.equal(strided, out)
        buf[:, 1:7, 16:144] = 7.0
        assert bool((buf == 7).all())


# ------------------------------------------------------------------ values
@pytest.mark.parametrize("dq,dc", TYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_masked_nan_and_inf_change_nothing(pkg, dq, dc, hd, bad):
    """Rows that do not see a key or value that is no finite number."""
    c = attn_case(11, [700, 210], [300, 210], 6, 2, hd, 64, dq, dc)
    first = torch.ones(c["q"].shape[0], dtype=torch.bool)
    clean = dict(c, k=c["k"].clone(), v=c["v"].clone())
    for b, slot, row0 in ((0, 613, 613 - 400), (1, 100, 300 + 100)):
        pg, off = c["tables"][b][slot // 64], slot % 64
        c["v"][pg, :, off, 5] = bad
        c["k"][pg, :, off, 9] = bad
        last = c["starts"][b + 1]
        first[row0:last] = False
    want = reference(clean)
    for wide in (False, True):
        out, lse = call(pkg, c, wide)
        check(clean, out, lse, rows=first, ref=want)
        assert not torch.isfinite(out[~first][0]).all()
        if wide and dq != F4:    # (bit by bit; in the other kernels a row's new maximum may move another's rounding)
            ref, ref_lse = call(pkg, clean, wide)
            assert torch.equal(out[first], ref[first]) and torch.equal(lse[first], ref_lse[first])


@pytest.mark.parametrize("dq,dc", TYPES)
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("down", [False, True])
def test_maxima_that_grow_along_the_cache(pkg, dq, dc, hd, down):
    c = attn_case(12, [1500, 260], [200, 260], 4, 2, hd, 64, dq, dc, q_scale=1.0)
    d = torch.nn.functional.normalize(torch.ones(hd, device="cuda"), dim=0)
    c["q"].copy_((c["q"].float() * 0.1 + (-6.0 if down else 6.0) * d).to(dq))
    for b in range(2):
        for s in range(c["lens"][b]):
            pg = c["tables"][b][s // 64]
            c["k"][pg, :, s % 64] = (c["k"][pg, :, s % 64].float() * 0.1 + d * (s / 16)).to(dc)
    both(pkg, c)


@pytest.mark.parametrize("dq,dc", TYPES)
def test_large_scores(pkg, dq, dc):
    c = attn_case(13, [400], [260], 4, 2, 128, 64, dq, dc, q_scale=60.0)
    both(pkg, c)


# ------------------------------------------------------------------ runs
@pytest.mark.parametrize("dq,dc", TYPES)
def test_same_result_in_every_run_and_on_another_stream(pkg, dq, dc):
    c = attn_case(14, [900, 300, 5], [400, 300, 5], 14, 2, 64, 16, dq, dc)
    a, la = call(pkg, c, True)
    tight = call(pkg, c)[0]
    for _ in range(4):
        b, lb = call(pkg, c, True)
        assert torch.equal(a, b) and torch.equal(la, lb) and torch.equal(tight, call(pkg, c)[0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out, lse = torch.full_like(a, 7.0), torch.full_like(la, 7.0)
    args = (c["q"], c["k"], c["v"], widened(c, True), i32(c["lens"]))
    starts = i32(c["starts"])
    torch.cuda.synchronize()
    pkg.chunk_attention(*args, starts=starts, max_rows=c["max_rows"], out=out, lse=lse, stream=st)
    st.synchronize()
    assert torch.equal(a, out) and torch.equal(la, lse)


def test_two_calls_at_once(pkg):
    cs = [attn_case(20 + i, [1200, 300], [500, 300], 14, 2, 64, 64) for i in range(2)]
    want = [call(pkg, c, True)[0] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    args = [dict(q=c["q"], k_cache=c["k"], v_cache=c["v"], tables=widened(c, True), lens=i32(c["lens"]),
                 starts=i32(c["starts"]), max_rows=c["max_rows"], out=torch.full_like(w, 7.0),
                 workspace=pkg.chunk_attention_workspace(c["q"], c["k"], None, c["max_rows"])) for c, w in zip(cs, want)]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, st in zip(args, streams):
            pkg.chunk_attention(**a, stream=st)
    torch.cuda.synchronize()
    for a, w in zip(args, want):
        assert torch.equal(a["out"], w)


def test_captured_and_replayed_with_other_lengths(pkg):
    c = attn_case(30, [900, 640], [333, 256], 6, 2, 128, 64)
    lens, starts = i32(c["lens"]), i32(c["starts"])
    out = torch.full_like(c["q"], 7.0)
    ws = pkg.chunk_attention_workspace(c["q"], c["k"], None, 400)
    args = dict(tables=widened(c, True), lens=lens, starts=starts, max_rows=400, out=out, workspace=ws)
    pkg.chunk_attention(c["q"], c["k"], c["v"], **args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.chunk_attention(c["q"], c["k"], c["v"], **args)
    for new_lens, new_starts in (([900, 640], [0, 333, 589]), ([700, 100], [0, 300, 400]), ([0, 64], [0, 0, 64])):
        lens.copy_(i32(new_lens))
        starts.copy_(i32(new_starts))
        out.fill_(7.0)
        ws.fill_(255)
        graph.replay()
        c["lens"], c["starts"] = new_lens, new_starts
        lse = call(pkg, c, True, max_rows=400)[1]
        check(c, out, lse)


@pytest.mark.parametrize("dt", [BF, FH])
@pytest.mark.parametrize("hd", [64, 128])
def test_long_contexts(pkg, dt, hd):
    lens = [40000] + [17000] * 7
    c = attn_case(40, lens, [40, 33, 1, 0, 20, 64, 5, 9], 8, 2, hd, 128, dt, dt, q_scale=1.0)
    both(pkg, c)


@pytest.mark.parametrize("dt", [BF, FH])
@pytest.mark.parametrize("hd", [64, 128])
def test_sums_that_move(pkg, dt, hd):
    """Beyond 16384 slots in one CTA output and sum move to the workspace. Some of
    the rows are compared: with them at the end of a shorter request."""
    m, n, g = 8192, 30000, 8
    c = attn_case(42, [n], [m], g, 1, hd, 128, dt, dt, q_scale=1.0)
    out, lse = call(pkg, c)
    for a, b in ((0, 20), (31, 33), (2111, 2140), (5000, 5001), (6500, 6520), (8160, 8192)):
        part = dict(c, q=c["q"][a:b], lens=[n - m + b], starts=[0, b - a])
        check(part, out[a:b], lse[a:b])


@pytest.mark.parametrize("hd,nkv,group,lens,rows", [
    (128, 4, 1, [40000], [3000]), (64, 16, 1, [40000], [2500]),
    (128, 2, 3, [30011, 7, 45000, 0, 25000], [3000, 7, 1500, 0, 2111]), (64, 8, 2, [30000, 41234], [2000, 1700])])
def test_rounds(pkg, hd, nkv, group, lens, rows):
    """More keys and values than L2 holds, and items that share them: two and
    three rounds. Some of the rows are compared, as above."""
    c = attn_case(43, lens, rows, nkv * group, nkv, hd, 128, BF, BF, q_scale=1.0)
    out, lse = call(pkg, c)
    for b, m in enumerate(rows):
        s0 = c["starts"][b]
        for a, e in ((0, 5), (m // 2 + 100, m // 2 + 103), (m - 6, m)):
            if not 0 <= a < e <= m:
                continue
            part = dict(c, q=c["q"][s0 + a:s0 + e], tables=[c["tables"][b]], lens=[lens[b] - m + e], starts=[0, e - a])
            check(part, out[s0 + a:s0 + e], lse[s0 + a:s0 + e])
    for _ in range(3):
        again = call(pkg, c)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    again = call(pkg, c, True)
    ends = torch.tensor(c["starts"][1:], device="cuda") - 1
    assert bool(torch.isfinite(again[0].float()).all()) and bool((again[0][ends].float() - out[ends].float()).abs().max() < 0.1)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("page", [16, 256])
def test_large_batches_of_prompts(pkg, hd, page):
    r = random.Random(hd)
    lens = [r.randint(1, 900) for _ in range(24)]
    rows = [r.choice([n, r.randint(1, n)]) for n in lens]
    c = attn_case(41, lens, rows, 7, 1, hd, page, BF, BF)
    both(pkg, c)


def test_offsets_past_32_bits(pkg):
    """Pages and rows whose elements lie more than 2^31 apart."""
    nkv, hd, page = 2, 128, 64
    pool = torch.empty((9, 2 ** 28 + 64), dtype=BF, device="cuda")
    k, v = (pool[:, o:o + nkv * page * hd].unflatten(1, (nkv, page, hd)) for o in (0, 2 ** 27))
    for x in (k, v):
        x.copy_(torch.randn(x.shape, device="cuda"))
    q = torch.empty((300, 2 ** 23), dtype=BF, device="cuda")[:, :4 * hd].unflatten(1, (4, hd))
    q.copy_(torch.randn(q.shape, device="cuda"))
    c = dict(q=q, k=k, v=v, tables=[[8, 3, 7, 1, 6, 0]], lens=[360], starts=[0, 300], max_rows=300)
    for wide in (False, True):
        out = torch.full((300, 2 ** 23), 7.0, dtype=BF, device="cuda")[:, :4 * hd].unflatten(1, (4, hd))
        res, lse = call(pkg, c, wide, out=out)
        check(c, res, lse)


@pytest.mark.parametrize("dq,dc", TYPES)
def test_workspace_of_any_contents_and_batches_of_other_sizes(pkg, dq, dc):
    """One workspace, full of ones, for calls of different sizes one after the other."""
    cs = [attn_case(44 + i, lens, rows, 6, 2, 128, 64, dq, dc)
          for i, (lens, rows) in enumerate([([900, 40, 2100], [300, 40, 700]), ([130], [130]), ([5000, 17], [60, 17])])]
    ws = pkg.chunk_attention_workspace(cs[0]["q"], cs[0]["k"], i32(cs[0]["tables"]), 700)
    ws.fill_(255)
    got = [(c, wide, *call(pkg, c, wide, workspace=ws)) for _ in range(2) for c in cs for wide in (False, True)]
    for i, (c, wide, out, lse) in enumerate(got):
        check(c, out, lse)
        ws.fill_(255 if i % 2 else 127)
        again = call(pkg, c, wide, workspace=ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_prior_calls_are_seen(pkg):
    """Append and chunk back to back: the attention waits for the cache."""
    c = attn_case(31, [1000], [600], 28, 4, 128, 64, pad=0)
    lens, starts, tables = i32(c["lens"]), i32(c["starts"]), i32(c["tables"])
    slots = torch.tensor([c["tables"][0][s // 64] * 64 + s % 64 for s in range(400, 1000)], dtype=torch.int32, device="cuda")
    for i in range(4):
        k, v = (torch.randn((600, 4, 128), dtype=BF, device="cuda") for _ in range(2))
        pkg.kv_append(k, v, slots, c["k"], c["v"])
        out = pkg.chunk_attention(c["q"], c["k"], c["v"], tables, lens, starts=starts, max_rows=600)
        again = pkg.chunk_attention(c["q"], c["k"], c["v"], tables, lens, starts=starts, max_rows=600)
        assert torch.equal(out, again)
    check(c, out, call(pkg, c)[1])


def test_refusals(pkg):
    c = attn_case(32, [200], [100], 4, 2, 64, 64)
    a = (c["q"], c["k"], c["v"], i32(c["tables"]), i32(c["lens"]))
    with pytest.raises(ValueError, match="max_rows"):
        pkg.chunk_attention(*a, starts=i32(c["starts"]))
    for kw in (dict(max_rows=0), dict(max_rows=2 ** 20 + 1), dict(scale=float("nan")), dict(scale=float("inf"))):
        with pytest.raises(pkg.SFError):
            pkg.chunk_attention(*a, starts=i32(c["starts"]), **{**dict(max_rows=100), **kw})
    with pytest.raises(ValueError, match="workspace"):
        pkg.chunk_attention(*a, starts=i32(c["starts"]), max_rows=100,
                            workspace=torch.empty(100, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pkg.SFError, match="overlap"):
        pkg.chunk_attention(*a, starts=i32(c["starts"]), max_rows=100, out=c["q"][:1].expand(c["q"].shape))
    with pytest.raises(pkg.SFError):
        pkg.chunk_attention(c["q"].half(), *a[1:], starts=i32(c["starts"]), max_rows=100)
    with pytest.raises(ValueError, match="requires grad"):
        pkg.chunk_attention(c["q"].clone().requires_grad_(), *a[1:], starts=i32(c["starts"]), max_rows=100)
