"""What the paged-cache operators refuse, at the C ABI and in the Python
wrappers, and the oracle's page plan against its own invariants. No GPU: a
refused call returns before anything is enqueued (its pointers are only
looked at for being null or misaligned)."""

import ctypes
import random

import pytest
import torch

from greedy_speculative_decoding_gb300 import _lib as L
from greedy_speculative_decoding_gb300 import build as B
from oracle import paged as op

PTR = 4096   # a non-null, well aligned address that a refused call never reads


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def cache(**kw):
    c = dict(k=PTR, v=PTR, dtype=L.SF_DT_BF16, n_pages=10, n_kv_heads=2, page=64, head_dim=64, reserved=0,
             k_page=8192, k_head=4096, k_slot=64, v_page=8192, v_head=4096, v_slot=64)
    c.update(kw)
    return L.PagedCache(**c)


def rows(heads, **kw):
    r = dict(data=PTR, dtype=L.SF_DT_BF16, n_heads=heads, row=heads * 64, head=64)
    r.update(kw)
    return L.Rows(**r)


BAD_CACHES = [
    (dict(k=None), L.SF_ERR_ARG), (dict(v=PTR + 8), L.SF_ERR_ARG), (dict(dtype=L.SF_DT_F32), L.SF_ERR_UNSUPPORTED),
    (dict(dtype=7), L.SF_ERR_UNSUPPORTED), (dict(head_dim=96), L.SF_ERR_UNSUPPORTED), (dict(page=48), L.SF_ERR_ARG),
    (dict(page=8), L.SF_ERR_ARG), (dict(page=512), L.SF_ERR_ARG), (dict(n_pages=0), L.SF_ERR_ARG),
    (dict(n_pages=2 ** 31 // 64), L.SF_ERR_ARG), (dict(n_kv_heads=0), L.SF_ERR_ARG), (dict(k_slot=68), L.SF_ERR_ARG),
    (dict(v_head=0), L.SF_ERR_ARG), (dict(k_page=-8192), L.SF_ERR_ARG), (dict(v_page=2048), L.SF_ERR_ARG),
]


def plan(lib, **kw):
    a = dict(lens=PTR, starts=PTR, batch=4, page=64, tables=PTR, width=8, held=PTR, free=PTR, capacity=100, n_free=PTR,
             n_rows=4, slots=PTR, positions=PTR, held_out=PTR, n_free_out=PTR, status=PTR)
    a.update(kw)
    return lib.sf_page_plan(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(lens=None), dict(starts=None), dict(tables=None), dict(held=None), dict(free=None), dict(n_free=None),
    dict(held_out=None), dict(n_free_out=None), dict(status=None), dict(batch=0), dict(batch=8193), dict(page=0),
    dict(page=24), dict(page=512), dict(width=0), dict(width=2 ** 30), dict(capacity=0), dict(capacity=2 ** 31 // 64),
    dict(n_rows=-1), dict(slots=None), dict(positions=None)])
def test_plan_refusals(lib, kw):
    assert plan(lib, **kw) == L.SF_ERR_ARG
    assert lib.sf_last_error()


def append(lib, c=None, n=3, k=None, v=None, slots=PTR, q=None, q_out=None, positions=None, rope=None, n_pos=0):
    r = ctypes.byref
    return lib.sf_kv_append(r(c or cache()), n, r(k or rows(2)), r(v or rows(2)), slots, r(q) if q else None,
                            r(q_out) if q_out else None, positions, rope, n_pos, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), L.SF_ERR_ARG), (dict(slots=None), L.SF_ERR_ARG), (dict(q=rows(4)), L.SF_ERR_ARG),
    (dict(q_out=rows(4)), L.SF_ERR_ARG), (dict(k=rows(3)), L.SF_ERR_ARG), (dict(v=rows(2, data=PTR + 2)), L.SF_ERR_ARG),
    (dict(k=rows(2, row=130)), L.SF_ERR_ARG), (dict(k=rows(2, head=68)), L.SF_ERR_ARG),
    (dict(k=rows(2, dtype=L.SF_DT_F32)), L.SF_ERR_UNSUPPORTED),
    (dict(k=rows(2, dtype=L.SF_DT_F16), v=rows(2, dtype=L.SF_DT_F16)), L.SF_ERR_UNSUPPORTED),
    (dict(q=rows(4, dtype=L.SF_DT_F32), q_out=rows(4)), L.SF_ERR_UNSUPPORTED),
    (dict(q=rows(4), q_out=rows(4, dtype=L.SF_DT_F32)), L.SF_ERR_ARG), (dict(q=rows(4), q_out=rows(5)), L.SF_ERR_ARG),
    (dict(rope=PTR, n_pos=4), L.SF_ERR_ARG), (dict(rope=PTR, positions=PTR, n_pos=0), L.SF_ERR_ARG),
    (dict(rope=PTR + 8, positions=PTR, n_pos=4), L.SF_ERR_ARG)])
def test_append_refusals(lib, kw, status):
    assert append(lib, **kw) == status
    assert lib.sf_last_error()


def attend(lib, c=None, q=None, out=None, n=3, tables=PTR, width=4, lens=PTR, starts=PTR, batch=3, max_rows=1,
           mask=None, scale=0.125, lse=None, ws=PTR):
    r = ctypes.byref
    return lib.sf_paged_attention(r(c or cache()), r(q or rows(4)), r(out or rows(4)), n, tables, width, lens, starts,
                                  batch, max_rows, mask, scale, lse, ws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), L.SF_ERR_ARG), (dict(batch=-1), L.SF_ERR_ARG), (dict(tables=None), L.SF_ERR_ARG),
    (dict(lens=None), L.SF_ERR_ARG), (dict(ws=None), L.SF_ERR_ARG), (dict(ws=PTR + 16), L.SF_ERR_ARG),
    (dict(q=rows(5), out=rows(5)), L.SF_ERR_ARG), (dict(out=rows(2)), L.SF_ERR_ARG),
    (dict(q=rows(4, dtype=L.SF_DT_F32)), L.SF_ERR_UNSUPPORTED),
    (dict(q=rows(4, dtype=L.SF_DT_F16), out=rows(4, dtype=L.SF_DT_F16)), L.SF_ERR_UNSUPPORTED),
    (dict(c=cache(dtype=L.SF_DT_F16), q=rows(4, dtype=L.SF_DT_F32), out=rows(4, dtype=L.SF_DT_F32)),
     L.SF_ERR_UNSUPPORTED),
    (dict(max_rows=0), L.SF_ERR_ARG), (dict(max_rows=81), L.SF_ERR_ARG), (dict(max_rows=65, mask=PTR), L.SF_ERR_ARG),
    (dict(starts=None, n=4), L.SF_ERR_ARG), (dict(starts=None, n=6), L.SF_ERR_ARG), (dict(width=0), L.SF_ERR_ARG),
    (dict(width=2 ** 30), L.SF_ERR_ARG), (dict(q=rows(4, data=PTR + 4)), L.SF_ERR_ARG),
    (dict(out=rows(4, row=260)), L.SF_ERR_ARG), (dict(scale=float("nan")), L.SF_ERR_ARG),
    (dict(scale=float("inf")), L.SF_ERR_ARG)])
def test_attention_refusals(lib, kw, status):
    assert attend(lib, **kw) == status
    assert lib.sf_last_error()


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_refusals(lib, kw, status):
    assert append(lib, c=cache(**kw)) == status
    assert attend(lib, c=cache(**kw)) == status


def test_nothing_to_do_is_ok(lib):
    assert append(lib, n=0) == L.SF_OK
    assert attend(lib, n=0) == L.SF_OK
    assert attend(lib, batch=0) == L.SF_OK


def test_rope_table_refusals(lib):
    for args in [(None, 4, 64, 1e4), (PTR + 4, 4, 64, 1e4), (PTR, 0, 64, 1e4), (PTR, 4, 63, 1e4), (PTR, 2 ** 30, 64, 1e4),
                 (PTR, 4, 64, 0.0), (PTR, 4, 64, float("inf"))]:
        assert lib.sf_rope_table(*args, None) == L.SF_ERR_ARG


def test_workspace_sizes(lib):
    f = lib.sf_paged_attention_workspace_bytes
    assert 0 < f(28, 4, 128, 9) <= 64 * 2 ** 20
    for bad in [(0, 1, 64, 1), (3, 2, 64, 1), (4, 2, 96, 1), (4, 2, 64, 0), (4, 2, 64, 81)]:
        assert f(*bad) == 0


@pytest.mark.parametrize("seed", range(6))
def test_oracle_plan_keeps_every_page_in_one_place(seed):
    r = random.Random(seed)
    B_, W, page, cap = r.randint(1, 9), 6, 16, 30
    pages = list(range(cap))
    r.shuffle(pages)
    tables, held = [[-1] * W for _ in range(B_)], [0] * B_
    free, n_free = pages, cap
    for _ in range(12):
        lens = [r.randint(0, W * page) if r.random() < 0.8 else 0 for _ in range(B_)]
        rows = [min(x, r.randint(0, 3)) for x in lens]
        starts = [sum(rows[:b]) for b in range(B_ + 1)]
        res = op.page_plan(lens, starts, tables, held, free, n_free, page, starts[-1] + 2)
        tables, held, free, n_free = res["tables"], res["held"], res["free"], res["n_free"]
        owned = [p for b in range(B_) for p in tables[b][:held[b]]] + free[:n_free]
        assert sorted(owned) == list(range(cap))
        used = [s for s in res["slots"] if s >= 0]
        assert len(used) == len(set(used))
        for b in range(B_):
            assert res["status"][b] == 1 or held[b] == -(-lens[b] // page)


@pytest.mark.parametrize("kw", [
    dict(row=0), dict(head=0), dict(row=32, head=512), dict(row=256, head=256), dict(row=64), dict(row=192, head=128),
    dict(row=-64)])
def test_rows_written_on_one_another(lib, kw):
    """Broadcast and overlapping outputs (three rows of four heads of 64)."""
    assert append(lib, q=rows(4), q_out=rows(4, **kw)) == L.SF_ERR_ARG
    assert attend(lib, out=rows(4, **kw)) == L.SF_ERR_ARG


@pytest.mark.parametrize("kw", [
    dict(k_slot=8, k_head=512), dict(k_head=64), dict(v_head=2048), dict(k_page=4096), dict(v_page=8184), dict(v=PTR)])
def test_cache_slots_written_on_one_another(lib, kw):
    """Two heads of 64 slots of 64 in a page; keys and values in one place."""
    c = cache(**{"v": 2 * PTR, **kw})
    assert append(lib, c=c) == L.SF_ERR_ARG
    assert b"overlap" in lib.sf_last_error() or b"are one" in lib.sf_last_error()


def test_overlap_is_told_exactly(lib):
    """Row layouts of every kind: refused exactly where two rows share an
    element (an allowed layout goes on to be refused for its scale)."""
    r = random.Random(3)
    seen = set()
    for _ in range(400):
        n, heads = r.randint(1, 5), r.choice([2, 4, 6])
        row, head = 8 * r.randint(0, 60), 8 * r.randint(0, 60)
        at = sorted(i * row + h * head for i in range(n) for h in range(heads))
        want = any(b - a < 64 for a, b in zip(at, at[1:]))
        seen.add(want)
        assert attend(lib, q=rows(heads), out=rows(heads, row=row, head=head), n=n, starts=PTR, batch=1,
                      scale=float("inf")) == L.SF_ERR_ARG
        assert (b"overlap" in lib.sf_last_error()) == want, (n, heads, row, head)
    assert seen == {False, True}


@pytest.fixture(scope="module")
def native():
    B.build()
    from greedy_speculative_decoding_gb300 import paged
    return paged._binding()


def plain_calls(native):
    """One call of each operator on CPU tensors: refused for that, if for nothing else (caches are looked at first)."""
    z = lambda *s, **kw: torch.zeros(s, **kw)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    return {
        "page_plan": (native.page_plan, [0, 0, 16, 3, i(2), i(3), i(2, 4), i(2), i(9), i(1), i(3), i(3), i(2), i(1), i(2)],
                      []),
        "kv_append": (native.kv_append, [0, 0, z(3, 2, 64), z(3, 2, 64), i(3), z(4, 2, 16, 64), z(4, 2, 16, 64),
                                         z(3, 4, 64), z(3, 4, 64), i(3), z(9, 32, 2)], [5, 6]),
        "paged_attention": (native.paged_attention, [0, 0, 1, None, z(3, 4, 64), z(4, 2, 16, 64), z(4, 2, 16, 64), i(2, 2),
                                                     i(2), i(3), None, z(3, 4, 64), None, i(9)], [5, 6]),
    }


@pytest.mark.parametrize("op", ["kv_append", "paged_attention"])
def test_tensors_that_require_grad(native, op):
    f, args, floats = plain_calls(native)[op]
    for k in floats:
        a = list(args)
        a[k] = a[k].clone().requires_grad_()
        with pytest.raises(ValueError, match="requires grad"):
            f(*a)
        with torch.no_grad(), pytest.raises(ValueError, match="on another device"):
            f(*a)


def test_binding_refuses_tensors_of_another_device(native):
    for f, args, _ in plain_calls(native).values():
        with pytest.raises(ValueError, match="on another device"):
            f(*args)
