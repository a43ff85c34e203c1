"""A key-value cache in pages: block tables and slot maps from request
lengths, RoPE and append, attention over the pages, and pages that several
requests hold. Argument marshalling over the C ABI, as in the engine's wrapper.

A pass over a batch of requests of different lengths runs the three in order
(``page_plan``, ``kv_append``, ``paged_attention``); what they need to know of
it lies on the device, so a captured pass can be replayed with other lengths.
``starts`` [B + 1] gives each request's token rows in the pass, ``lens`` [B]
its tokens including them. ``chunk_attention`` takes the attention's place for
prompts and long pieces of them.

Requests that continue one another share pages: ``page_fork``, ``page_free``
and ``page_compact`` change tables, counts and the stack of free pages, and
``page_copy`` moves what the first and the last of them say in every layer.
``shares`` int32 [n_pages] counts a page's holders beyond the first (zeros to
begin with).

Every call takes tensors of the current CUDA device and enqueues its work on
``stream`` (default: the current stream). Tensors that a call allocates itself
belong to that stream. The calls have no gradients: tensors that require grad
are refused unless gradients are off.
"""

import importlib
from typing import NamedTuple

import torch

from . import _lib as L

_native = None


def _binding():
    """The extension module that checks and marshals the tensors (csrc/paged_py.cpp)."""
    global _native
    if _native is None:
        L.load()
        _native = importlib.import_module(__package__ + "._paged")
    return _native


class PagePlan(NamedTuple):
    """What page_plan leaves: each row's cache slot and position, the pages
    held by each request, the free pages, and each request's status (0 served,
    1 not enough pages, 2 refused)."""
    slots: torch.Tensor
    positions: torch.Tensor
    held: torch.Tensor
    n_free: torch.Tensor
    status: torch.Tensor


def _device(stream):
    """(current device, stream handle)."""
    dev = torch._C._cuda_getDevice()
    return dev, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _empty(shape, dtype, dev, stream):
    """A tensor that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def page_plan(lens, starts, tables, held, free, n_free, page, n_rows=None, slots=None, positions=None, held_out=None,
              n_free_out=None, status=None, stream=None) -> PagePlan:
    """Block tables and slot maps from request lengths (sf_page_plan): pages
    that requests no longer need go back onto the stack of free pages, pages
    that they lack are taken from it, and each of the n_rows token rows gets
    its cache slot and position.

    lens int32 [B], starts int32 [B + 1], tables int32 [B, W] (updated in
    place), held int32 [B], free int32 [capacity] (the stack, updated in
    place), n_free int32 [1]. held and n_free are updated in place unless
    held_out and n_free_out are given; slots and positions int32 [n_rows] and
    status int32 [B] are allocated unless given."""
    call = (_native or _binding()).page_plan
    dev, st = _device(stream)
    if n_rows is None:
        given = slots if slots is not None else positions
        if given is None:
            raise ValueError("n_rows is needed unless slots or positions are given")
        n_rows = given.shape[0]
    if slots is None:
        slots = _empty(n_rows, torch.int32, dev, stream)
    if positions is None:
        positions = _empty(n_rows, torch.int32, dev, stream)
    if status is None:
        status = _empty(tables.shape[0], torch.int32, dev, stream)
    if held_out is None:
        held_out = held
    if n_free_out is None:
        n_free_out = n_free
    s = call(dev, st, page, n_rows, lens, starts, tables, held, free, n_free, slots, positions, held_out, n_free_out,
             status)
    if s:
        L.check(s)
    return PagePlan(slots, positions, held_out, n_free_out, status)


def rope_table(n_pos: int, head_dim: int, theta: float, stream=None) -> torch.Tensor:
    """The engine's RoPE table (sf_rope_table): fp32 [n_pos, head_dim // 2, 2],
    (cos, sin) of pos * theta ** (-2 i / head_dim)."""
    dev, st = _device(stream)
    out = _empty((n_pos, head_dim // 2, 2), torch.float32, dev, stream)
    L.check(L.load().sf_rope_table(out.data_ptr(), n_pos, head_dim, theta, st))
    return out


def kv_append(k, v, slots, k_cache, v_cache, q=None, q_out=None, positions=None, rope=None, stream=None):
    """RoPE and cache append (sf_kv_append): rows k, v [n, kv_heads, head_dim]
    into the cache slots slots int32 [n] (negative: a padding row, for which
    nothing is written); with rope (rope_table's layout) k and q are rotated by
    positions int32 [n] first. Returns q_out (allocated in the cache's type
    unless given; its padding rows are then undefined), or None without q."""
    call = (_native or _binding()).kv_append
    dev, st = _device(stream)
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
    elif q_out is None:
        q_out = _empty(q.shape, k_cache.dtype, dev, stream)
    if rope is not None and positions is None:
        raise ValueError("rope without positions")
    s = call(dev, st, k, v, slots, k_cache, v_cache, q, q_out, positions, rope)
    if s:
        L.check(s)
    return q_out


def paged_attention_workspace(q, k_cache, tables, max_rows: int) -> torch.Tensor:
    """Scratch for paged_attention calls with these head counts and at most
    max_rows rows a request. Any contents will do; calls that may overlap on
    the GPU (on two streams, or in two graphs) need one each."""
    return torch.empty(_workspace_bytes(q, k_cache, max_rows), dtype=torch.uint8, device=q.device)


def _workspace_bytes(q, k_cache, max_rows):
    n = L.load().sf_paged_attention_workspace_bytes(q.shape[1], k_cache.shape[1], k_cache.shape[3], max_rows)
    if n == 0:
        raise L.SFError(L.SF_ERR_ARG, "sf_paged_attention_workspace_bytes rejected the heads, head_dim or max_rows")
    return n


def paged_attention(q, k_cache, v_cache, tables, lens, starts=None, max_rows=None, mask=None, scale=None, out=None,
                    lse=None, workspace=None, stream=None) -> torch.Tensor:
    """Attention of each request's newest rows over its pages
    (sf_paged_attention): q [n, heads, head_dim], tables int32 [B, W], lens
    int32 [B] (tokens including the pass's rows), starts int32 [B + 1] (the
    rows of request b are starts[b] .. starts[b + 1] - 1, at most max_rows;
    None: n / B rows each). A row sees everything before the pass's rows, and
    of these up to itself, or with mask (int64 [n]) the rows whose bit is set.
    scale defaults to 1 / sqrt(head_dim). out (q's type) and workspace are
    allocated unless given; lse float32 [n, heads] is written when given.
    Rows outside every request are left as they were."""
    call = (_native or _binding()).paged_attention
    dev, st = _device(stream)
    if max_rows is None:
        if starts is not None:
            raise ValueError("max_rows is needed with starts")
        max_rows = max(1, q.shape[0] // max(1, tables.shape[0]))
    if out is None:
        out = _empty(q.shape, q.dtype, dev, stream)
    if workspace is None:
        workspace = _empty(_workspace_bytes(q, k_cache, max_rows), torch.uint8, dev, stream)
    s = call(dev, st, max_rows, scale, q, k_cache, v_cache, tables, lens, starts, mask, out, lse, workspace)
    if s:
        L.check(s)
    return out


def chunk_attention_workspace(q, k_cache, tables, max_rows: int) -> torch.Tensor:
    """Scratch for chunk_attention calls with these head counts and at most
    max_rows rows a request. Any contents will do; calls that may overlap on
    the GPU (on two streams, or in two graphs) need one each."""
    return torch.empty(_chunk_bytes(q, k_cache, max_rows), dtype=torch.uint8, device=q.device)


def _chunk_bytes(q, k_cache, max_rows):
    n = L.load().sf_chunk_attention_workspace_bytes(q.shape[1], k_cache.shape[1], k_cache.shape[3], max_rows)
    if n == 0:
        raise L.SFError(L.SF_ERR_ARG, "sf_chunk_attention_workspace_bytes rejected the heads, head_dim or max_rows")
    return n


def chunk_attention(q, k_cache, v_cache, tables, lens, starts=None, max_rows=None, scale=None, out=None, lse=None,
                    workspace=None, stream=None) -> torch.Tensor:
    """Attention of a chunk of new tokens over the pages (sf_chunk_attention):
    as paged_attention without a mask, for requests of up to 2^20 rows. q [n,
    heads, head_dim]; row j of request b's n_b rows sees its slots 0 ..
    lens[b] - n_b + j. max_rows (needed with starts): the most rows of one
    request. Rows outside every request are left as they were."""
    call = (_native or _binding()).chunk_attention
    dev, st = _device(stream)
    if max_rows is None:
        if starts is not None:
            raise ValueError("max_rows is needed with starts")
        max_rows = max(1, q.shape[0] // max(1, tables.shape[0]))
    if out is None:
        out = _empty(q.shape, q.dtype, dev, stream)
    if workspace is None:
        workspace = _empty(_chunk_bytes(q, k_cache, max_rows), torch.uint8, dev, stream)
    s = call(dev, st, max_rows, scale, q, k_cache, v_cache, tables, lens, starts, None, out, lse, workspace)
    if s:
        L.check(s)
    return out


class PageFork(NamedTuple):
    """What page_fork leaves for page_copy: page source[i] to be copied into
    target[i], its first slots[i] slots (-1, -1, 0: nothing), and each fork's
    status (0 forked, 1 not enough pages, 2 refused)."""
    source: torch.Tensor
    target: torch.Tensor
    slots: torch.Tensor
    status: torch.Tensor


class PageMoves(NamedTuple):
    """What page_compact leaves: the new tables and shares, and for page_copy
    the count pairs of pages, source[i] to be copied into target[i]."""
    tables: torch.Tensor
    shares: torch.Tensor
    source: torch.Tensor
    target: torch.Tensor
    count: torch.Tensor


def page_free(requests, tables, held, shares, free, n_free, page, keep=None, status=None, stream=None) -> torch.Tensor:
    """Requests cut short or ended (sf_page_free): requests[i] keeps the pages
    of its first keep[i] tokens (None: none). Pages that nobody else holds go
    onto the stack. requests and keep int32 [n]; tables, held, shares, free and
    n_free are updated in place. Returns status int32 [n]: 0, or 2 where the
    request was refused and left as it is."""
    call = (_native or _binding()).page_free
    dev, st = _device(stream)
    if status is None:
        status = _empty(requests.shape, torch.int32, dev, stream)
    s = call(dev, st, page, requests, keep, tables, held, shares, free, n_free, status)
    if s:
        L.check(s)
    return status


def page_fork(src, dst, lens, tables, held, shares, free, n_free, page, source=None, target=None, slots=None,
              status=None, stream=None) -> PageFork:
    """Requests forked (sf_page_fork): dst[i], which holds nothing, shares the
    full pages of src[i]'s first lens[src[i]] tokens and gets a page off the
    stack for the rest, whose contents page_copy brings. src and dst int32 [n],
    lens int32 [B]; tables, held, shares and n_free are updated in place;
    source, target, slots and status int32 [n] are allocated unless given."""
    call = (_native or _binding()).page_fork
    dev, st = _device(stream)
    if source is None:
        source = _empty(src.shape, torch.int32, dev, stream)
    if target is None:
        target = _empty(src.shape, torch.int32, dev, stream)
    if slots is None:
        slots = _empty(src.shape, torch.int32, dev, stream)
    if status is None:
        status = _empty(src.shape, torch.int32, dev, stream)
    s = call(dev, st, page, src, dst, lens, tables, held, shares, free, n_free, source, target, slots, status)
    if s:
        L.check(s)
    return PageFork(source, target, slots, status)


def page_compact(tables, held, shares, free, n_free, tables_out=None, shares_out=None, source=None, target=None,
                 count=None, stream=None) -> PageMoves:
    """The held pages moved to the lowest numbers (sf_page_compact). tables and
    shares are updated in place unless tables_out and shares_out are given;
    free and n_free are written anew: every page that no table holds counts as
    free. source and target int32 [n_pages // 2] at least and count int32 [1]
    are allocated unless given."""
    call = (_native or _binding()).page_compact
    dev, st = _device(stream)
    if tables_out is None:
        tables_out = tables
    if shares_out is None:
        shares_out = shares
    if source is None:
        source = _empty(shares.shape[0] // 2, torch.int32, dev, stream)
    if target is None:
        target = _empty(shares.shape[0] // 2, torch.int32, dev, stream)
    if count is None:
        count = _empty(1, torch.int32, dev, stream)
    s = call(dev, st, tables, held, shares, tables_out, shares_out, free, n_free, source, target, count)
    if s:
        L.check(s)
    return PageMoves(tables_out, shares_out, source, target, count)


def page_copy(source, target, k_cache, v_cache, slots=None, count=None, stream=None):
    """Pages copied (sf_page_copy): page source[i] into page target[i], or its
    first slots[i] slots, for the first count pairs (int32 [1] on the device;
    None: all). Caches [pages, kv_heads, page, head_dim] of one layer, or
    [layers, pages, kv_heads, page, head_dim]: every layer is copied. Pairs
    with a negative number are passed over."""
    call = (_native or _binding()).page_copy
    dev, st = _device(stream)
    s = call(dev, st, source, target, k_cache, v_cache, slots, count)
    if s:
        L.check(s)
