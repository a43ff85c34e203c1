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

import ctypes
import math
import struct
from typing import NamedTuple

import torch

from . import _lib as L

_DT = {torch.float32: L.SF_DT_F32, torch.bfloat16: L.SF_DT_BF16, torch.float16: L.SF_DT_F16}
# sf_paged_cache and sf_rows as bytes (their fields as in L.PagedCache and L.Rows).
_CACHE, _ROWS = struct.Struct("=QQiiiiiiqqqqqq"), struct.Struct("=Qiiqq")
assert _CACHE.size == ctypes.sizeof(L.PagedCache) and _ROWS.size == ctypes.sizeof(L.Rows)


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
    dev = torch.cuda.current_device()
    return dev, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _empty(shape, dtype, dev, stream):
    """A tensor that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _ptr(name, t, shape, dtype, dev):
    """The address of a contiguous tensor, checked."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {tuple(shape)} on cuda:{dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(name, t, n, hd, dev):
    dt = _DT.get(t.dtype)
    if dt is None or t.dim() != 3 or t.get_device() != dev:
        raise ValueError(f"{name}: expected rows [{n}, heads, {hd}] (fp32, bf16 or fp16) on cuda:{dev}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    (rows, heads, d), (s0, s1, s2) = t.shape, t.stride()
    if rows != n or d != hd or s2 != 1:
        raise ValueError(f"{name}: expected rows [{n}, heads, {hd}] with the last dimension contiguous, got "
                         f"{tuple(t.shape)} with strides {t.stride()}")
    return _ROWS.pack(t.data_ptr(), dt, heads, s0, s1)


def _cache(k, v, dev):
    """(sf_paged_cache, kv_heads, head_dim)."""
    if k.dim() != 4 or k.shape != v.shape or k.dtype is not v.dtype or k.dtype not in _DT:
        raise ValueError(f"caches: expected k and v [pages, kv_heads, page, head_dim] of one type, got "
                         f"{k.dtype} {tuple(k.shape)} and {v.dtype} {tuple(v.shape)}")
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError(f"caches: expected tensors on cuda:{dev}, got {k.device} and {v.device}")
    (k0, k1, k2, k3), (v0, v1, v2, v3), (p, h, s, d) = k.stride(), v.stride(), k.shape
    if k3 != 1 or v3 != 1:
        raise ValueError("caches: the last dimension must be contiguous")
    return _CACHE.pack(k.data_ptr(), v.data_ptr(), _DT[k.dtype], p, h, s, d, 0, k0, k1, k2, v0, v1, v2), h, d


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
    dev, st = _device(stream)
    if tables.dim() != 2 or free.dim() != 1:
        raise ValueError("tables must be [B, W], free [capacity]")
    (B, W), (cap,), i32 = tables.shape, free.shape, torch.int32
    if n_rows is None:
        given = slots if slots is not None else positions
        if given is None:
            raise ValueError("n_rows is needed unless slots or positions are given")
        n_rows = given.shape[0]
    if slots is None:
        slots = _empty(n_rows, i32, dev, stream)
    if positions is None:
        positions = _empty(n_rows, i32, dev, stream)
    if status is None:
        status = _empty(B, i32, dev, stream)
    held_out = held if held_out is None else held_out
    n_free_out = n_free if n_free_out is None else n_free_out
    b1, n1 = (B,), (n_rows,)
    s = lib.sf_page_plan(
        _ptr("lens", lens, b1, i32, dev), _ptr("starts", starts, (B + 1,), i32, dev), B, page,
        _ptr("tables", tables, (B, W), i32, dev), W, _ptr("held", held, b1, i32, dev),
        _ptr("free", free, (cap,), i32, dev), cap, _ptr("n_free", n_free, (1,), i32, dev), n_rows,
        _ptr("slots", slots, n1, i32, dev), _ptr("positions", positions, n1, i32, dev),
        _ptr("held_out", held_out, b1, i32, dev), _ptr("n_free_out", n_free_out, (1,), i32, dev),
        _ptr("status", status, b1, i32, dev), st)
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
    lib = L.load()
    dev, st = _device(stream)
    cache, _, hd = _cache(k_cache, v_cache, dev)
    n = k.shape[0]
    rq = ro = pos = cs = None
    n_pos = 0
    if q is not None:
        if q_out is None:
            q_out = _empty(q.shape, k_cache.dtype, dev, stream)
        rq, ro = _rows("q", q, n, hd, dev), _rows("q_out", q_out, n, hd, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if rope is not None:
        if positions is None:
            raise ValueError("rope without positions")
        n_pos = rope.shape[0]
        pos = _ptr("positions", positions, (n,), torch.int32, dev)
        cs = _ptr("rope", rope, (n_pos, hd // 2, 2), torch.float32, dev)
    s = lib.sf_kv_append(cache, n, _rows("k", k, n, hd, dev), _rows("v", v, n, hd, dev),
                         _ptr("slots", slots, (n,), torch.int32, dev), rq, ro, pos, cs, n_pos, st)
    if s:
        L.check(s)
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
    dev, st = _device(stream)
    cache, nkv, hd = _cache(k_cache, v_cache, dev)
    if tables.dim() != 2:
        raise ValueError("tables must be [B, W]")
    n, nq, (B, W), i32 = q.shape[0], q.shape[1], tables.shape, torch.int32
    if max_rows is None:
        if starts is not None:
            raise ValueError("max_rows is needed with starts")
        max_rows = max(1, n // max(1, B))
    if out is None:
        out = _empty(q.shape, q.dtype, dev, stream)
    need = lib.sf_paged_attention_workspace_bytes(nq, nkv, hd, max_rows)
    if workspace is None:
        workspace = _empty(need, torch.uint8, dev, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous() or workspace.nbytes < need:
        raise ValueError(f"workspace: expected {need} contiguous bytes on cuda:{dev}")
    s = lib.sf_paged_attention(
        cache, _rows("q", q, n, hd, dev), _rows("out", out, n, hd, dev), n, _ptr("tables", tables, (B, W), i32, dev), W,
        _ptr("lens", lens, (B,), i32, dev), None if starts is None else _ptr("starts", starts, (B + 1,), i32, dev), B,
        max_rows, None if mask is None else _ptr("mask", mask, (n,), torch.int64, dev),
        1.0 / math.sqrt(hd) if scale is None else scale,
        None if lse is None else _ptr("lse", lse, (n, nq), torch.float32, dev), workspace.data_ptr(), st)
    if s:
        L.check(s)
    return out
