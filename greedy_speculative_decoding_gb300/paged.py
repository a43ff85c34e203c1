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
belong to that stream.
"""

import contextlib
import ctypes
import math
from typing import NamedTuple

import torch

from . import _lib as L

_DT = {torch.float32: L.SF_DT_F32, torch.bfloat16: L.SF_DT_BF16, torch.float16: L.SF_DT_F16}


class PagePlan(NamedTuple):
    """What page_plan leaves: each row's cache slot and position, the pages
    held by each request, the free pages, and each request's status (0 served,
    1 not enough pages, 2 refused)."""
    slots: torch.Tensor
    positions: torch.Tensor
    held: torch.Tensor
    n_free: torch.Tensor
    status: torch.Tensor


def _stream(stream):
    """(stream handle, context to allocate in): tensors made for a call on
    another stream than the current one must belong to it."""
    cur = torch.cuda.current_stream()
    if stream is None or stream.cuda_stream == cur.cuda_stream:
        return ctypes.c_void_p(cur.cuda_stream), contextlib.nullcontext()
    return ctypes.c_void_p(stream.cuda_stream), torch.cuda.stream(stream)


def _on_gpu(dev, **tensors):
    """Refuse tensors that are not on the current CUDA device."""
    for name, t in tensors.items():
        if t is not None and (not t.is_cuda or t.device.index != dev):
            raise ValueError(f"{name}: expected a tensor on cuda:{dev}, got {t.device}")


def _ints(name, t, shape, dtype=torch.int32):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _rows(name, t, n, hd):
    if t.dtype not in _DT or t.dim() != 3 or t.shape[0] != n or t.shape[2] != hd or t.stride(2) != 1:
        raise ValueError(f"{name}: expected rows [{n}, heads, {hd}] (fp32, bf16 or fp16, last dimension contiguous), "
                         f"got {t.dtype} {tuple(t.shape)}")
    return L.Rows(t.data_ptr(), _DT[t.dtype], t.shape[1], t.stride(0), t.stride(1))


def _cache(k, v):
    if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.dtype not in _DT:
        raise ValueError(f"caches: expected k and v [pages, kv_heads, page, head_dim] of one type, got "
                         f"{k.dtype} {tuple(k.shape)} and {v.dtype} {tuple(v.shape)}")
    ks, vs = k.stride(), v.stride()
    if ks[3] != 1 or vs[3] != 1:
        raise ValueError("caches: the last dimension must be contiguous")
    p, h, s, d = k.shape
    return L.PagedCache(k.data_ptr(), v.data_ptr(), _DT[k.dtype], p, h, s, d, 0, ks[0], ks[1], ks[2], vs[0], vs[1], vs[2])


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
    lib = L.load()
    dev = torch.cuda.current_device()
    _on_gpu(dev, lens=lens, starts=starts, tables=tables, held=held, free=free, n_free=n_free, slots=slots,
            positions=positions, held_out=held_out, n_free_out=n_free_out, status=status)
    if tables.dim() != 2 or free.dim() != 1:
        raise ValueError("tables must be [B, W], free [capacity]")
    B, W = tables.shape
    if n_rows is None:
        given = slots if slots is not None else positions
        if given is None:
            raise ValueError("n_rows is needed unless slots or positions are given")
        n_rows = given.shape[0]
    st, own = _stream(stream)
    with own:
        if slots is None:
            slots = torch.empty(n_rows, dtype=torch.int32, device=lens.device)
        if positions is None:
            positions = torch.empty(n_rows, dtype=torch.int32, device=lens.device)
        if status is None:
            status = torch.empty(B, dtype=torch.int32, device=lens.device)
    held_out = held if held_out is None else held_out
    n_free_out = n_free if n_free_out is None else n_free_out
    L.check(lib.sf_page_plan(
        _ints("lens", lens, (B,)), _ints("starts", starts, (B + 1,)), B, page, _ints("tables", tables, (B, W)), W,
        _ints("held", held, (B,)), _ints("free", free, free.shape), free.shape[0], _ints("n_free", n_free, (1,)),
        n_rows, _ints("slots", slots, (n_rows,)), _ints("positions", positions, (n_rows,)),
        _ints("held_out", held_out, (B,)), _ints("n_free_out", n_free_out, (1,)), _ints("status", status, (B,)), st))
    return PagePlan(slots, positions, held_out, n_free_out, status)


def rope_table(n_pos: int, head_dim: int, theta: float, stream=None) -> torch.Tensor:
    """The engine's RoPE table (sf_rope_table): fp32 [n_pos, head_dim // 2, 2],
    (cos, sin) of pos * theta ** (-2 i / head_dim)."""
    st, own = _stream(stream)
    with own:
        out = torch.empty((n_pos, head_dim // 2, 2), dtype=torch.float32, device="cuda")
    L.check(L.load().sf_rope_table(out.data_ptr(), n_pos, head_dim, theta, st))
    return out


def kv_append(k, v, slots, k_cache, v_cache, q=None, q_out=None, positions=None, rope=None, stream=None):
    """RoPE and cache append (sf_kv_append): rows k, v [n, kv_heads, head_dim]
    into the cache slots slots int32 [n] (negative: a padding row, for which
    nothing is written); with rope (rope_table's layout) k and q are rotated by
    positions int32 [n] first. Returns q_out (allocated in the cache's type
    unless given; its padding rows are then undefined), or None without q."""
    lib = L.load()
    dev = torch.cuda.current_device()
    _on_gpu(dev, k=k, v=v, slots=slots, k_cache=k_cache, v_cache=v_cache, q=q, q_out=q_out, positions=positions,
            rope=rope)
    cache = _cache(k_cache, v_cache)
    n, hd = k.shape[0], cache.head_dim
    st, own = _stream(stream)
    rq = ro = None
    if q is not None:
        if q_out is None:
            with own:
                q_out = torch.empty(q.shape, dtype=k_cache.dtype, device=q.device)
        rq, ro = _rows("q", q, n, hd), _rows("q_out", q_out, n, hd)
    elif q_out is not None:
        raise ValueError("q_out without q")
    pos = cs = None
    n_pos = 0
    if rope is not None:
        if positions is None or rope.dim() != 3 or rope.shape[1:] != (hd // 2, 2) or rope.dtype != torch.float32 \
                or not rope.is_contiguous():
            raise ValueError(f"rope: expected positions and a contiguous fp32 table [n_pos, {hd // 2}, 2]")
        pos, cs, n_pos = _ints("positions", positions, (n,)), rope.data_ptr(), rope.shape[0]
    rk, rv = _rows("k", k, n, hd), _rows("v", v, n, hd)
    L.check(lib.sf_kv_append(ctypes.byref(cache), n, ctypes.byref(rk), ctypes.byref(rv),
                             _ints("slots", slots, (n,)), None if rq is None else ctypes.byref(rq),
                             None if ro is None else ctypes.byref(ro), pos, cs, n_pos, st))
    return q_out


def paged_attention_workspace(q, k_cache, tables, max_rows: int) -> torch.Tensor:
    """Scratch for paged_attention calls with these head counts and at most
    max_rows rows a request. Any contents will do; calls that may overlap on
    the GPU (on two streams, or in two graphs) need one each."""
    n = L.load().sf_paged_attention_workspace_bytes(q.shape[1], k_cache.shape[1], k_cache.shape[3], max_rows)
    if n == 0:
        raise L.SFError(L.SF_ERR_ARG, "sf_paged_attention_workspace_bytes rejected the heads, head_dim or max_rows")
    return torch.empty(n, dtype=torch.uint8, device=q.device)


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
    lib = L.load()
    dev = torch.cuda.current_device()
    _on_gpu(dev, q=q, k_cache=k_cache, v_cache=v_cache, tables=tables, lens=lens, starts=starts, mask=mask, out=out,
            lse=lse, workspace=workspace)
    cache = _cache(k_cache, v_cache)
    if tables.dim() != 2:
        raise ValueError("tables must be [B, W]")
    n, hd = q.shape[0], cache.head_dim
    B, W = tables.shape
    if max_rows is None:
        if starts is not None:
            raise ValueError("max_rows is needed with starts")
        max_rows = max(1, n // max(1, B))
    st, own = _stream(stream)
    with own:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if workspace is None:
            workspace = paged_attention_workspace(q, k_cache, tables, max_rows)
    need = lib.sf_paged_attention_workspace_bytes(q.shape[1], k_cache.shape[1], hd, max_rows)
    if not workspace.is_contiguous() or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace: expected {need} contiguous bytes")
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != tuple(q.shape[:2])
                            or not lse.is_contiguous()):
        raise ValueError(f"lse: expected a contiguous float32 tensor {tuple(q.shape[:2])}")
    rq, ro = _rows("q", q, n, hd), _rows("out", out, n, hd)
    L.check(lib.sf_paged_attention(
        ctypes.byref(cache), ctypes.byref(rq), ctypes.byref(ro), n, _ints("tables", tables, (B, W)), W,
        _ints("lens", lens, (B,)), None if starts is None else _ints("starts", starts, (B + 1,)), B, max_rows,
        None if mask is None else _ints("mask", mask, (n,), torch.int64),
        1.0 / math.sqrt(hd) if scale is None else scale, None if lse is None else lse.data_ptr(),
        workspace.data_ptr(), st))
    return out
