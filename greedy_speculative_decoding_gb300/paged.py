"""A key-value cache in pages: block tables and slot maps from request
lengths, RoPE and append, and attention over the pages. Argument marshalling
over the C ABI, as in the engine's wrapper.

A pass over a batch of requests of different lengths runs the three in order
(``page_plan``, ``kv_append``, ``paged_attention``); what they need to know of
it lies on the device, so a captured pass can be replayed with other lengths.
``starts`` [B + 1] gives each request's token rows in the pass, ``lens`` [B]
its tokens including them.

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
