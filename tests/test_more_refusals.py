"""What chunk_attention, the operators of shared pages and token_logprobs refuse
at the C ABI, and the oracle's shared pages against their own invariants. No
GPU: a refused call returns before anything is enqueued."""

import ctypes
import random

import pytest

from greedy_speculative_decoding_gb300 import _lib as L
from oracle import paged as op
from test_paged_refusals import BAD_CACHES, PTR, cache, lib, rows  # noqa: F401


def chunk(lib, c=None, q=None, out=None, n=300, tables=PTR, width=8, lens=PTR, starts=PTR, batch=3, max_rows=200,
          scale=0.125, lse=None, ws=PTR):
    r = ctypes.byref
    return lib.sf_chunk_attention(r(c or cache()), r(q or rows(4)), r(out or rows(4)), n, tables, width, lens, starts,
                                  batch, max_rows, scale, lse, ws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), L.SF_ERR_ARG), (dict(batch=-1), L.SF_ERR_ARG), (dict(tables=None), L.SF_ERR_ARG),
    (dict(lens=None), L.SF_ERR_ARG), (dict(ws=None), L.SF_ERR_ARG), (dict(ws=PTR + 16), L.SF_ERR_ARG),
    (dict(q=rows(5), out=rows(5)), L.SF_ERR_ARG), (dict(out=rows(2)), L.SF_ERR_ARG),
    (dict(q=rows(4, dtype=L.SF_DT_F32)), L.SF_ERR_UNSUPPORTED),
    (dict(q=rows(4, dtype=L.SF_DT_F16), out=rows(4, dtype=L.SF_DT_F16)), L.SF_ERR_UNSUPPORTED),
    (dict(c=cache(dtype=L.SF_DT_F16), q=rows(4, dtype=L.SF_DT_F32), out=rows(4, dtype=L.SF_DT_F32)),
     L.SF_ERR_UNSUPPORTED),
    (dict(max_rows=0), L.SF_ERR_ARG), (dict(max_rows=2 ** 20 + 1), L.SF_ERR_ARG),
    (dict(q=rows(4096), out=rows(4096), c=cache(n_kv_heads=1), max_rows=2 ** 20), L.SF_ERR_UNSUPPORTED),
    (dict(starts=None, n=301), L.SF_ERR_ARG), (dict(starts=None, n=900), L.SF_ERR_ARG), (dict(width=0), L.SF_ERR_ARG),
    (dict(width=2 ** 30), L.SF_ERR_ARG), (dict(q=rows(4, data=PTR + 4)), L.SF_ERR_ARG),
    (dict(out=rows(4, row=260)), L.SF_ERR_ARG), (dict(out=rows(4, row=0)), L.SF_ERR_ARG),
    (dict(scale=float("nan")), L.SF_ERR_ARG), (dict(scale=float("inf")), L.SF_ERR_ARG)])
def test_chunk_refusals(lib, kw, status):
    assert chunk(lib, **kw) == status
    assert b"sf_chunk_attention" in lib.sf_last_error()


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_refusals(lib, kw, status):
    assert chunk(lib, c=cache(**kw)) == status
    assert copy(lib, c=cache(**kw)) == status


def free(lib, requests=PTR, keep=None, n=3, batch=4, page=16, tables=PTR, width=8, held=PTR, shares=PTR, n_pages=50,
         stack=PTR, capacity=50, n_free=PTR, status=PTR):
    return lib.sf_page_free(requests, keep, n, batch, page, tables, width, held, shares, n_pages, stack, capacity,
                            n_free, status, None)


def fork(lib, src=PTR, dst=PTR, n=3, lens=PTR, batch=4, page=16, tables=PTR, width=8, held=PTR, shares=PTR, n_pages=50,
         stack=PTR, capacity=50, n_free=PTR, source=PTR, target=PTR, slots=PTR, status=PTR):
    return lib.sf_page_fork(src, dst, n, lens, batch, page, tables, width, held, shares, n_pages, stack, capacity,
                            n_free, source, target, slots, status, None)


def compact(lib, tables=PTR, batch=4, width=8, held=PTR, shares=PTR, n_pages=50, tables_out=PTR, shares_out=PTR,
            stack=PTR, capacity=50, n_free=PTR, source=PTR, target=PTR, moves=25, count=PTR):
    return lib.sf_page_compact(tables, batch, width, held, shares, n_pages, tables_out, shares_out, stack, capacity,
                               n_free, source, target, moves, count, None)


def copy(lib, c=None, layers=2, k_layer=81920, v_layer=81920, source=PTR, target=PTR, slots=None, n=3, count=None):
    return lib.sf_page_copy(ctypes.byref(c or cache(v=2 * PTR)), layers, k_layer, v_layer, source, target, slots, n,
                            count, None)


LIST = [dict(n=-1), dict(n=8193), dict(batch=0), dict(batch=8193), dict(page=0), dict(page=24), dict(page=512),
        dict(width=0), dict(width=2 ** 26 + 1), dict(batch=8192, width=2 ** 17), dict(n=8192, width=2 ** 17, batch=1),
        dict(n_pages=0), dict(capacity=0), dict(tables=None), dict(held=None), dict(shares=None), dict(stack=None),
        dict(n_free=None), dict(status=None)]


@pytest.mark.parametrize("kw", LIST + [dict(requests=None)])
def test_free_refusals(lib, kw):
    assert free(lib, **kw) == L.SF_ERR_ARG and b"sf_page_free" in lib.sf_last_error()


@pytest.mark.parametrize("kw", LIST + [dict(src=None), dict(dst=None), dict(lens=None), dict(source=None),
                                       dict(target=None), dict(slots=None)])
def test_fork_refusals(lib, kw):
    assert fork(lib, **kw) == L.SF_ERR_ARG and b"sf_page_fork" in lib.sf_last_error()


@pytest.mark.parametrize("kw,status", [(kw, L.SF_ERR_ARG) for kw in (
    dict(batch=0), dict(batch=8193), dict(width=0), dict(batch=8192, width=2 ** 17), dict(n_pages=0), dict(capacity=49),
    dict(moves=24), dict(tables=None), dict(held=None), dict(shares=None), dict(tables_out=None), dict(shares_out=None),
    dict(stack=None), dict(n_free=None), dict(source=None), dict(target=None), dict(count=None))]
    + [(dict(n_pages=2 ** 20 + 1, capacity=2 ** 21, moves=2 ** 20), L.SF_ERR_UNSUPPORTED)])
def test_compact_refusals(lib, kw, status):
    assert compact(lib, **kw) == status and b"sf_page_compact" in lib.sf_last_error()


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(layers=0), dict(layers=2 ** 23 + 1), dict(source=None), dict(target=None), dict(k_layer=0),
    dict(v_layer=-8), dict(k_layer=81924), dict(v_layer=81912), dict(k_layer=2 ** 39), dict(layers=3, k_layer=8192),
    dict(c=cache()), dict(c=cache(v=2 * PTR, k_slot=8)), dict(c=cache(v=2 * PTR, v_page=4096))])
def test_copy_refusals(lib, kw):
    assert copy(lib, **kw) == L.SF_ERR_ARG and b"sf_page_copy" in lib.sf_last_error()


def apart(names):
    """An address of its own for each array, 256 KB apart."""
    return {name: PTR + (i << 18) for i, name in enumerate(names)}


FREE = ("requests", "keep", "tables", "held", "shares", "stack", "n_free", "status")
FORK = ("src", "dst", "lens", "tables", "held", "shares", "stack", "n_free", "source", "target", "slots", "status")
COMPACT = ("tables", "held", "shares", "tables_out", "shares_out", "stack", "n_free", "source", "target", "count")


@pytest.mark.parametrize("f,names,written,allowed", [
    (free, FREE, {"held", "shares", "stack", "n_free", "status"}, ()),
    (fork, FORK, {"tables", "held", "shares", "n_free", "source", "target", "slots", "status"}, ()),
    (compact, COMPACT, {"tables_out", "shares_out", "stack", "n_free", "source", "target", "count"},
     ({"tables", "tables_out"}, {"shares", "shares_out"}))])
def test_written_arrays_over_others_are_refused(lib, f, names, written, allowed):
    ints = dict(requests=3, keep=3, status=3, src=3, dst=3, source=3, target=3, slots=3, tables=32, tables_out=32, held=4,
                lens=4, shares=50, shares_out=50, stack=50, n_free=1, count=1)
    if f is compact:
        ints.update(source=25, target=25)
    for x in names:
        for y in names:
            if x == y or not {x, y} & written:
                continue
            for shift in (0, 4 * ints[y] - 4) if {x, y} not in allowed else (4,):   # (up to its last element)
                kw = apart(names)
                kw[x] = kw[y] + shift
                assert f(lib, **kw) == L.SF_ERR_ARG and b"overlaps" in lib.sf_last_error(), (x, y, shift)


def score(lib, logits=PTR, dtype=L.SF_DT_F32, row=100, n=3, vocab=100, tokens=PTR, top=5):
    return lib.sf_token_logprobs(logits, dtype, row, n, vocab, tokens, top, PTR, PTR, PTR, PTR, PTR, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), L.SF_ERR_ARG), (dict(vocab=0), L.SF_ERR_ARG), (dict(vocab=2 ** 31 - 1), L.SF_ERR_ARG),
    (dict(top=-1), L.SF_ERR_ARG), (dict(top=33), L.SF_ERR_ARG), (dict(top=5, vocab=4), L.SF_ERR_ARG),
    (dict(logits=None), L.SF_ERR_ARG), (dict(tokens=None), L.SF_ERR_ARG), (dict(logits=PTR + 2), L.SF_ERR_ARG),
    (dict(logits=PTR + 1, dtype=L.SF_DT_BF16), L.SF_ERR_ARG), (dict(row=-1), L.SF_ERR_ARG),
    (dict(row=2 ** 39), L.SF_ERR_ARG), (dict(dtype=3), L.SF_ERR_UNSUPPORTED), (dict(dtype=-1), L.SF_ERR_UNSUPPORTED)])
def test_logprob_refusals(lib, kw, status):
    assert score(lib, **kw) == status and b"sf_token_logprobs" in lib.sf_last_error()


def test_outputs_over_other_arrays_are_refused(lib):
    """3 rows of 100 fp32 logits, 100 apart; five of top."""
    bytes = [1200, 12, 12, 12, 12, 60, 60]                 # logits, tokens, outputs
    for x in range(2, 7):
        for y in range(7):
            if x == y:
                continue
            for shift in (0, bytes[y] - 4):
                at = [PTR + (i << 18) for i in range(7)]
                at[x] = at[y] + shift
                assert lib.sf_token_logprobs(at[0], L.SF_DT_F32, 100, 3, 100, at[1], 5, *at[2:], None) == L.SF_ERR_ARG
                assert b"overlaps" in lib.sf_last_error(), (x, y, shift)


def test_nothing_to_do_is_ok(lib):
    assert chunk(lib, n=0) == chunk(lib, batch=0) == L.SF_OK
    assert free(lib, n=0, requests=None) == fork(lib, n=0, src=None) == copy(lib, n=0) == score(lib, n=0) == L.SF_OK


def test_workspace_sizes(lib):
    f = lib.sf_chunk_attention_workspace_bytes
    assert 0 < f(28, 4, 128, 16411) == f(28, 4, 128, 2 ** 20) <= 128 * 2 ** 20
    for bad in [(0, 1, 64, 1), (3, 2, 64, 1), (4, 2, 96, 1), (4, 2, 64, 0), (4, 2, 64, 2 ** 20 + 1)]:
        assert f(*bad) == 0


@pytest.mark.parametrize("seed", range(20))
def test_oracle_counts_every_holder(seed):
    r = random.Random(seed)
    B, W, page = r.randint(2, 9), r.randint(1, 6), 16
    held, lens, n = [0] * B, [0] * B, r.randint(5, 40)
    P = n
    tables, shares, stack = [[-1] * W for _ in range(B)], [0] * n, list(range(n))
    for _ in range(12):
        x = op.page_fork([r.randrange(-1, B + 1) for _ in range(5)], [r.randrange(-1, B + 1) for _ in range(5)], lens,
                         tables, held, shares, stack, n, page)
        tables, held, shares, n = x["tables"], x["held"], x["shares"], x["n_free"]
        lens = [min(max(a, h * page - 3 if h else 0), h * page) for a, h in zip(lens, held)]
        more = [min(W * page, a + r.randint(0, 30)) for a in lens]
        y = op.page_plan(more, [0] * (B + 1), tables, held, stack, n, page, 0)
        lens = [a if s == 0 else b for a, b, s in zip(more, lens, y["status"])]
        tables, held, stack, n = y["tables"], y["held"], y["free"], y["n_free"]
        q = [r.randrange(-1, B + 1) for _ in range(4)]
        z = op.page_free(q, [r.choice([0, 0, r.randint(0, 60)]) for _ in q], tables, held, shares, stack, n, page)
        held, shares, stack, n = z["held"], z["shares"], z["free"], z["n_free"]
        lens = [min(a, h * page) for a, h in zip(lens, held)]
        count = [0] * P
        for t, h in zip(tables, held):
            for p in t[:h]:
                count[p] += 1
        assert [max(c - 1, 0) for c in count] == shares
        assert sorted(stack[:n]) == [p for p in range(P) if not count[p]]
