"""PyTorch-facing wrappers of rotary positions and the paged key/value cache
(zl_rope_*, zl_paged_* and zl_pages_* in include/zl_attn.h).

Tensors: q [T, H, d], k and v [T, Hk, d] (bf16, rope also float32), with heads
and columns contiguous and any distance between tokens, so that they may be
parts of one projection's rows.  A layer's pools are k_pages and v_pages
[P, Hk, page, d] bf16; page_table [S, cols], kv_lens [S] and page_refs [P] are
int32 tensors on the same device.  kv_lens counts the new tokens of a call.
cu_seqlens are host sequences of ints, or host_int32 of one.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import _lib
from .attention import _check_like, _check_tensor, _workspace_bytes, alloc_workspace

_BF16, _I32 = torch.bfloat16, torch.int32


def host_int32(values) -> _lib.HostInt32:
    """A cu_seqlens list as the library takes it, made once for many calls."""
    return _lib.HostInt32(values)


def _cu(values):
    if not isinstance(values, _lib.HostInt32):
        values = _lib.HostInt32(values)
    if values.last is None:
        raise ValueError("cu_seqlens must have at least one entry")
    return values


def _on_stream(fn):
    """Runs fn under the stream it is given, so that what it allocates belongs
    to that stream too."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, stream=stream, **kw)
    return call


class _On:
    """Makes the tensors' device the current one while the library is called
    (its launches go there) and gives that device's current stream."""
    __slots__ = ("index", "guard")

    def __init__(self, tensor, stream):
        self.index = tensor.device.index
        if stream is not None and stream.device_index != self.index:
            raise ValueError(f"the stream belongs to device {stream.device_index}, the tensors to {self.index}")
        self.guard = None if self.index == torch.cuda.current_device() else torch.cuda.device(self.index)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _check_rows(t, name, tokens, heads, dim, dtype, device):
    """[tokens, heads, dim] with contiguous heads and columns."""
    if t.shape != (tokens, heads, dim) or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be {(tokens, heads, dim)} {dtype} on {device}, "
                         f"got {tuple(t.shape)} {t.dtype} on {t.device}")
    if tokens and heads and (t.stride(2) != 1 or (heads > 1 and t.stride(1) != dim)):
        raise ValueError(f"{name}: a token's heads and columns must be contiguous")


def _row_stride(t):
    """Elements between tokens (one token may have any)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def _check_int32(t, name, shape, device):
    _check_like(t, name, shape, _I32, device)


def _require_cuda(*tensors):
    for t in tensors:
        if not t.is_cuda:
            raise ValueError("tensors must be CUDA tensors")


# ------------------------------------------------------------------ rotary positions
class RopePlan:
    """Frequencies and layout of rotary positions (zl_rope_t), made once.

    axes        rotated columns of each position axis, even (default: all of
                head_dim on one axis); their sum may be less than head_dim
    base        frequency base: pair j of an axis of d columns has base^(-2j/d)
    interleaved pairs are neighbours (2i, 2i+1) instead of halves (i, i + r/2)
    factor      every frequency is divided by it (positions scaled down) ...
    ramp        ... or, with (low, high, length), only those that turn less
                than `low` times over `length` positions, the ones that turn
                more than `high` times stay, and those between are blended
    magnitude   factor of the result
    """

    def __init__(self, head_dim, axes=None, base=10000.0, interleaved=False, factor=1.0, ramp=None, magnitude=1.0):
        axes = (int(head_dim),) if axes is None else tuple(int(a) for a in axes)
        self.struct = _lib.Rope()
        self.n_axes = len(axes)
        self.head_dim = int(head_dim)
        arr, n = _lib.int32_array(axes)
        ramp_arr = None if ramp is None else (ctypes.c_double * 3)(*(float(x) for x in ramp))
        _lib.check(_lib.load().zl_rope_init(ctypes.byref(self.struct), self.head_dim, int(bool(interleaved)), n, arr,
                                            float(base), float(factor), ramp_arr, float(magnitude)), "zl_rope_init")


def _positions(positions, plan, tokens, device):
    """Pointer and distance between axes of positions [T] or [n_axes, T]."""
    if positions.dtype != _I32 or positions.device != device:
        raise ValueError(f"positions must be int32 on {device}")
    if positions.shape != (plan.n_axes, tokens) and not (plan.n_axes == 1 and positions.shape == (tokens,)):
        raise ValueError(f"positions must be [{plan.n_axes}, {tokens}], got {tuple(positions.shape)}")
    if tokens > 1 and positions.stride(-1) != 1:
        raise ValueError("positions must be contiguous along the tokens")
    return positions.data_ptr(), (positions.stride(0) if plan.n_axes > 1 else tokens)


def _overlap(a, b):
    """Whether two row tensors share memory without being the same rows."""
    if a.numel() == 0 or b.numel() == 0 or (a.data_ptr() == b.data_ptr() and a.stride() == b.stride()
                                            and a.shape == b.shape):
        return False
    if a.untyped_storage().data_ptr() != b.untyped_storage().data_ptr():
        return False
    ends = []
    for t in (a, b):
        first = t.data_ptr()
        row = t.shape[1] * t.shape[2] * t.element_size()
        ends.append((first, first + (t.shape[0] - 1) * _row_stride(t) * t.element_size() + row, row,
                     _row_stride(t) * t.element_size()))
    (a0, a1, ra, sa), (b0, b1, rb, sb) = ends
    if a1 <= b0 or b1 <= a0:
        return False
    if sa == sb:        # columns of the same rows: apart when their offsets within a row are
        d = (b0 - a0) % sa
        return not (d >= ra and d + rb <= sa)
    return True


def _rope(name, q, k, positions, plan, q_out, k_out, stream):
    lib = _lib.load()
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q and k must be [T, heads, d]")
    if q.dtype not in (_BF16, torch.float32):
        raise TypeError(f"unsupported dtype {q.dtype}")
    tokens, nq, hd = q.shape
    if hd != plan.head_dim:
        raise ValueError(f"the plan is for head_dim {plan.head_dim}, q has {hd}")
    _check_rows(q, "q", tokens, nq, hd, q.dtype, q.device)
    nk = 0
    if k is not None:
        nk = k.shape[1]
        _check_rows(k, "k", tokens, nk, hd, q.dtype, q.device)
    elif k_out is not None:
        raise ValueError("k_out without k")
    pos, pos_stride = _positions(positions, plan, tokens, q.device)
    if q_out is None:
        q_out = torch.empty((tokens, nq, hd), dtype=q.dtype, device=q.device)
    if k is not None and k_out is None:
        k_out = torch.empty((tokens, nk, hd), dtype=q.dtype, device=q.device)
    _check_rows(q_out, "q_out", tokens, nq, hd, q.dtype, q.device)
    outs = [q_out]
    if k is not None:
        _check_rows(k_out, "k_out", tokens, nk, hd, q.dtype, q.device)
        outs.append(k_out)
    for i, o in enumerate(outs):
        for t in (q,) if k is None else (q, k):
            if _overlap(o, t):
                raise ValueError("an output overlaps an input without being it")
        if i and (_overlap(o, outs[0]) or (o.numel() and o.data_ptr() == outs[0].data_ptr())):
            raise ValueError("q_out and k_out overlap")
    if tokens == 0:
        return q_out, k_out
    _require_cuda(q)
    code = _lib.ZL_BF16 if q.dtype == _BF16 else _lib.ZL_FP32
    with _On(q, stream) as s:
        st = getattr(lib, name)(ctypes.byref(plan.struct), q.data_ptr(), _row_stride(q),
                                0 if k is None else k.data_ptr(), 0 if k is None else _row_stride(k), pos, pos_stride,
                                tokens, nq, nk, code, q_out.data_ptr(), _row_stride(q_out),
                                0 if k is None else k_out.data_ptr(), 0 if k is None else _row_stride(k_out), s)
    _lib.check(st, name)
    return q_out, k_out


@_on_stream
def rope_fwd(q, k, positions, plan, q_out=None, k_out=None, stream=None):
    """Turns q [T, Hq, d] and k [T, Hk, d] (or None) by their tokens' positions
    (int32 [T], or [n_axes, T]).  Returns (q_out, k_out); an output may be its
    own input."""
    return _rope("zl_rope_fwd", q, k, positions, plan, q_out, k_out, stream)


@_on_stream
def rope_bwd(dq, dk, positions, plan, dq_out=None, dk_out=None, stream=None):
    """Gradient of rope_fwd: from the gradients of its outputs to those of its
    inputs.  Returns (dq_out, dk_out)."""
    return _rope("zl_rope_bwd", dq, dk, positions, plan, dq_out, dk_out, stream)


# ------------------------------------------------------------------ the cache
def _cache(k_pages, v_pages, page_table, kv_lens, seqs):
    if k_pages.dim() != 4 or page_table.dim() != 2:
        raise ValueError("k_pages must be [P, Hk, page, d] and page_table [S, cols]")
    dev = k_pages.device
    _check_like(v_pages, "v_pages", k_pages.shape, k_pages.dtype, dev)
    if k_pages.dtype != _BF16:
        raise TypeError("the pages must be bf16")
    if page_table.shape[0] != seqs:
        raise ValueError(f"page_table has {page_table.shape[0]} rows, the batch {seqs} sequences")
    _check_int32(page_table, "page_table", page_table.shape, dev)
    _check_int32(kv_lens, "kv_lens", (seqs,), dev)
    if not (k_pages.is_contiguous() and v_pages.is_contiguous() and page_table.is_contiguous()
            and kv_lens.is_contiguous()):
        raise ValueError("pages, page_table and kv_lens must be contiguous")
    p, nk, page, hd = k_pages.shape
    return _lib.PagedCache(k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), kv_lens.data_ptr(),
                           page_table.shape[1], p, page, nk, hd, 0)


@_on_stream
def paged_append(k, v, k_pages, v_pages, page_table, kv_lens, cu_seqlens, q=None, q_out=None, rope=None,
                 positions=None, stream=None):
    """Writes a batch's new tokens k, v [T, Hk, d] into the pages: sequence s's
    rows of cu_seqlens become its last positions below kv_lens[s].  With a
    RopePlan the keys (and q [T, H, d], if given) are turned at their cache
    positions, or at `positions`.  Returns the turned q (or None)."""
    lib = _lib.load()
    cu = _cu(cu_seqlens)
    cache = _cache(k_pages, v_pages, page_table, kv_lens, len(cu) - 1)
    tokens, dev = cu.last, k_pages.device
    _check_rows(k, "k", tokens, cache.num_kv_heads, cache.head_dim, _BF16, dev)
    _check_rows(v, "v", tokens, cache.num_kv_heads, cache.head_dim, _BF16, dev)
    nq = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [T, H, d]")
        nq = q.shape[1]
        _check_rows(q, "q", tokens, nq, cache.head_dim, _BF16, dev)
        if q_out is None:
            q_out = torch.empty((tokens, nq, cache.head_dim), dtype=_BF16, device=dev)
        _check_rows(q_out, "q_out", tokens, nq, cache.head_dim, _BF16, dev)
        for t in (q, k, v):
            if _overlap(q_out, t) or (t is not q and q_out.numel() and q_out.data_ptr() == t.data_ptr()):
                raise ValueError("q_out overlaps an input without being q")
    elif q_out is not None:
        raise ValueError("q_out without q")
    pos, pos_stride = 0, 0
    if positions is not None:
        if rope is None:
            raise ValueError("positions without a rope plan")
        pos, pos_stride = _positions(positions, rope, tokens, dev)
    _require_cuda(k_pages)
    if tokens == 0:
        return q_out
    with _On(k_pages, stream) as s:
        st = lib.zl_paged_append(ctypes.byref(cache), k.data_ptr(), _row_stride(k), v.data_ptr(), _row_stride(v),
                                 cu.array, len(cu) - 1, None if rope is None else ctypes.byref(rope.struct), pos,
                                 pos_stride, 0 if not nq else q.data_ptr(), 0 if not nq else _row_stride(q), nq,
                                 0 if not nq else q_out.data_ptr(), 0 if not nq else _row_stride(q_out), s)
    _lib.check(st, "zl_paged_append")
    return q_out


def paged_attn_workspace_bytes(cu_seqlens_q, max_kv_len, num_heads, num_kv_heads, head_dim) -> int:
    lib = _lib.load()
    cu = _cu(cu_seqlens_q)
    out = ctypes.c_size_t(0)
    _lib.check(lib.zl_paged_attn_workspace_size(cu.array, len(cu) - 1, max_kv_len, num_heads, num_kv_heads, head_dim,
                                                ctypes.byref(out)), "zl_paged_attn_workspace_size")
    return int(out.value)


@_on_stream
def paged_attn(q, k_pages, v_pages, page_table, kv_lens, cu_seqlens_q, max_kv_len, causal=True, window=0,
               softmax_scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of each sequence's new queries q [Tq, H, d] over its cached
    keys and values.  The queries stand at the last positions below kv_lens;
    max_kv_len (host) bounds kv_lens.  Returns (o [Tq, H, d], lse [H, Tq])."""
    lib = _lib.load()
    cu = _cu(cu_seqlens_q)
    cache = _cache(k_pages, v_pages, page_table, kv_lens, len(cu) - 1)
    if q.dim() != 3:
        raise ValueError("q must be [Tq, H, d]")
    tq, nh, hd = q.shape
    if tq != cu.last:
        raise ValueError(f"q has {tq} rows, cu_seqlens_q ends at {cu.last}")
    dev = q.device
    _check_rows(q, "q", tq, nh, cache.head_dim, _BF16, k_pages.device)
    if out is None:
        out = torch.empty((tq, nh, hd), dtype=_BF16, device=dev)
    else:
        _check_like(out, "out", (tq, nh, hd), _BF16, dev)
    if lse is None:
        lse = torch.empty((nh, tq), dtype=torch.float32, device=dev)
    else:
        _check_like(lse, "lse", (nh, tq), torch.float32, dev)
    if not (out.is_contiguous() and lse.is_contiguous()):
        raise ValueError("out and lse must be contiguous")
    _require_cuda(q)
    if workspace is None:
        workspace = alloc_workspace(paged_attn_workspace_bytes(cu, max_kv_len, nh, cache.num_kv_heads, hd), dev)
    scale = 1.0 / math.sqrt(hd) if softmax_scale is None else float(softmax_scale)
    with _On(q, stream) as s:
        st = lib.zl_paged_attn(ctypes.byref(cache), q.data_ptr(), _row_stride(q), cu.array, len(cu) - 1, max_kv_len,
                               nh, scale, int(bool(causal)), int(window), out.data_ptr(), lse.data_ptr(),
                               0 if workspace is None else workspace.data_ptr(), _workspace_bytes(workspace), s)
    _lib.check(st, "zl_paged_attn")
    return out, lse


# ------------------------------------------------------------------ whole pages
def _tables(page_table, kv_lens, page_refs, page_size):
    if page_table.dim() != 2 or page_refs.dim() != 1:
        raise ValueError("page_table must be [S, cols] and page_refs [P]")
    dev = page_table.device
    _check_int32(page_table, "page_table", page_table.shape, dev)
    _check_int32(kv_lens, "kv_lens", (page_table.shape[0],), dev)
    _check_int32(page_refs, "page_refs", page_refs.shape, dev)
    if not (page_table.is_contiguous() and kv_lens.is_contiguous() and page_refs.is_contiguous()):
        raise ValueError("page_table, kv_lens and page_refs must be contiguous")
    _require_cuda(page_table)
    return _lib.PageTables(page_table.data_ptr(), kv_lens.data_ptr(), page_refs.data_ptr(), page_table.shape[0],
                           page_table.shape[1], page_refs.shape[0], page_size)


def _pool(cache, num_pages=None, device=None):
    """cache [..., P, Hk, page, d] with contiguous pages; the dimensions before
    P (layers, keys and values) are the groups."""
    if cache.dim() < 4:
        raise ValueError("the cache must be [..., P, Hk, page, d]")
    p, nk, page, hd = cache.shape[-4:]
    if num_pages is not None and p != num_pages:
        raise ValueError(f"the cache has {p} pages, page_refs {num_pages}")
    if device is not None and cache.device != device:
        raise ValueError(f"the cache must be on {device}")
    if not cache.is_contiguous():
        raise ValueError("the cache must be contiguous")
    _require_cuda(cache)
    size = nk * page * hd * cache.element_size()
    groups = cache.numel() // max(1, p * nk * page * hd)
    return _lib.PagePool(cache.data_ptr(), size, p * size, groups, p)


def _list(t, name, device):
    if t.dim() != 1:
        raise ValueError(f"{name} must be a vector")
    _check_int32(t, name, t.shape, device)
    _check_tensor(t, name)
    return t.shape[0]


def _status(status, device):
    if status is None:
        return torch.empty(1, dtype=_I32, device=device)
    _check_int32(status, "status", (1,), device)
    return status


def pages_workspace_bytes(num_pages) -> int:
    out = ctypes.c_size_t(0)
    _lib.check(_lib.load().zl_pages_workspace_size(num_pages, ctypes.byref(out)), "zl_pages_workspace_size")
    return int(out.value)


@_on_stream
def pages_extend(page_table, kv_lens, page_refs, counts, page_size, status=None, stream=None):
    """Makes room for counts[s] (int32, device) new tokens in every slot, in
    place: kv_lens grows, free pages (lowest first) enter the rows.  Returns a
    device int32 [1]: 0, or the pages lacking, or -1 for counts that are
    negative or do not fit a row; unless it is 0 nothing was changed."""
    t = _tables(page_table, kv_lens, page_refs, page_size)
    _check_int32(counts, "counts", kv_lens.shape, kv_lens.device)
    _check_tensor(counts, "counts")
    status = _status(status, kv_lens.device)
    with _On(kv_lens, stream) as s:
        st = _lib.load().zl_pages_extend(ctypes.byref(t), counts.data_ptr(), status.data_ptr(), s)
    _lib.check(st, "zl_pages_extend")
    return status


@_on_stream
def pages_fork(cache, page_table, kv_lens, page_refs, parents, children, status=None, workspace=None, stream=None):
    """Makes each empty slot children[i] a copy of slot parents[i] (int32,
    device), in place: full pages are shared, a part-filled last page is copied
    in every group of cache [..., P, Hk, page, d].  Returns a device int32 [1]
    as pages_extend does."""
    t = _tables(page_table, kv_lens, page_refs, cache.shape[-2] if cache.dim() >= 2 else 0)
    p = _pool(cache, page_refs.shape[0], page_table.device)
    n = _list(parents, "parents", kv_lens.device)
    if _list(children, "children", kv_lens.device) != n:
        raise ValueError("parents and children differ in length")
    status = _status(status, kv_lens.device)
    if workspace is None:
        workspace = alloc_workspace(pages_workspace_bytes(page_refs.shape[0]), kv_lens.device)
    with _On(kv_lens, stream) as s:
        st = _lib.load().zl_pages_fork(ctypes.byref(p), ctypes.byref(t), parents.data_ptr(), children.data_ptr(), n,
                                       status.data_ptr(), workspace.data_ptr(), _workspace_bytes(workspace), s)
    _lib.check(st, "zl_pages_fork")
    return status


@_on_stream
def pages_free(page_table, kv_lens, page_refs, slots, page_size, stream=None):
    """Empties the slots (int32, device), in place."""
    t = _tables(page_table, kv_lens, page_refs, page_size)
    n = _list(slots, "slots", kv_lens.device)
    with _On(kv_lens, stream) as s:
        st = _lib.load().zl_pages_free(ctypes.byref(t), slots.data_ptr(), n, s)
    _lib.check(st, "zl_pages_free")


@_on_stream
def pages_compact(cache, page_table, kv_lens, page_refs, live=None, workspace=None, stream=None):
    """Moves the used pages to the front of the pool, in place, in every group
    of cache [..., P, Hk, page, d].  Returns their number, a device int32 [1]."""
    t = _tables(page_table, kv_lens, page_refs, cache.shape[-2] if cache.dim() >= 2 else 0)
    p = _pool(cache, page_refs.shape[0], page_table.device)
    live = _status(live, kv_lens.device)
    if workspace is None:
        workspace = alloc_workspace(pages_workspace_bytes(page_refs.shape[0]), kv_lens.device)
    with _On(kv_lens, stream) as s:
        st = _lib.load().zl_pages_compact(ctypes.byref(p), ctypes.byref(t), live.data_ptr(), workspace.data_ptr(),
                                          _workspace_bytes(workspace), s)
    _lib.check(st, "zl_pages_compact")
    return live


@_on_stream
def pages_copy(cache, src, dst, stream=None):
    """Copies page src[i] over page dst[i] (int32, device) in every group of
    cache [..., P, Hk, page, d]; no page may be both, nor a target twice."""
    p = _pool(cache)
    n = _list(src, "src", cache.device)
    if _list(dst, "dst", cache.device) != n:
        raise ValueError("src and dst differ in length")
    with _On(cache, stream) as s:
        st = _lib.load().zl_pages_copy(ctypes.byref(p), src.data_ptr(), dst.data_ptr(), n, s)
    _lib.check(st, "zl_pages_copy")
