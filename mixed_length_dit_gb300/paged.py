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
import math
import struct

import torch

from . import _lib
from .attention import _check_like

_BF16, _I32 = torch.bfloat16, torch.int32


# The structs of the C ABI that a call fills, packed in one step (a call on a
# single token is bound by the host).
_CACHE = struct.Struct("@4P6i")          # zl_paged_cache_t
_TABLES = struct.Struct("@3P4i")         # zl_page_tables_t
_POOL = struct.Struct("@P2q2i")          # zl_page_pool_t


def host_int32(values) -> _lib.HostInt32:
    """A cu_seqlens list as the library takes it, made once for many calls."""
    return _lib.HostInt32(values)


def _cu(values):
    if not isinstance(values, _lib.HostInt32):
        values = _lib.HostInt32(values)
    if values.n == 0:
        raise ValueError("cu_seqlens must have at least one entry")
    return values


def _short(name, *args):
    """The call by the compiled binding, if all is as it should be: its result;
    None if the long way has to be taken."""
    r = getattr(_lib._bind or _lib.bind(), name)(*args)
    if type(r) is int:
        _lib.check(r, "zl_" + _NAMES[name])
    return r


_NAMES = {"rope": "rope", "append": "paged_append", "append_after": "paged_append_ex", "attn": "paged_attn", "extend": "pages_extend",
          "fork": "pages_fork", "compact": "pages_compact"}


def _int32(value, name):
    """ctypes keeps the low 32 bits of a larger number."""
    if not -2**31 <= value < 2**31:
        raise ValueError(f"{name} must fit 32 bits, got {value}")


def _call(name, index, stream, *args):
    """Calls the library with the device `index` of the call's tensors as the
    current one (its launches go there) and that device's current stream."""
    if index < 0:
        raise ValueError("tensors must be CUDA tensors")
    fn = getattr(_lib.load(), name)
    if stream is not None:
        if stream.device_index != index:
            raise ValueError(f"the stream belongs to device {stream.device_index}, the tensors to {index}")
    elif torch._C._cuda_getDevice() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
        if st:
            _lib.check(st, name)
        return
    with torch.cuda.device(index):
        _lib.check(fn(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream), name)


def _empty(like, shape, dtype, stream):
    """A new tensor on the device of `like`; it belongs to the stream that the
    call is given."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _rows(t, name, tokens, heads, dim, dtype, device):
    """Checks for [tokens, heads, dim] with contiguous heads and columns;
    returns the elements between tokens (for one token, any do)."""
    if t.shape != (tokens, heads, dim) or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name} must be {(tokens, heads, dim)} {dtype} on {device}, "
                         f"got {tuple(t.shape)} {t.dtype} on {t.device}")
    s0, s1, s2 = t.stride()
    if tokens and heads and (s2 != 1 or (heads > 1 and s1 != dim)):
        raise ValueError(f"{name}: a token's heads and columns must be contiguous")
    return s0 if tokens > 1 else heads * dim


def _exact(t, name, shape, dtype, device):
    """Checks for this shape, dtype and device, contiguous."""
    if t.shape != shape or t.dtype is not dtype or t.device != device:
        _check_like(t, name, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _scratch(workspace, device):
    """Pointer and size of a workspace (or None)."""
    if workspace is None:
        return 0, 0
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


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
        self._point()

    def _point(self):
        self.ref = ctypes.byref(self.struct)
        self.address = ctypes.addressof(self.struct)

    def __reduce__(self):
        # copies and pickles point at a struct of their own
        return _plan_of, (bytes(self.struct),)


def _plan_of(data):
    plan = RopePlan.__new__(RopePlan)
    plan.struct = _lib.Rope.from_buffer_copy(data)
    plan.n_axes, plan.head_dim = plan.struct.n_axes, plan.struct.head_dim
    plan._point()
    return plan


def _positions(positions, plan, tokens, device):
    """Pointer and distance between axes of positions [T] or [n_axes, T]."""
    if positions.dtype is not _I32 or positions.device != device:
        raise ValueError(f"positions must be int32 on {device}")
    if positions.shape != (plan.n_axes, tokens) and not (plan.n_axes == 1 and positions.shape == (tokens,)):
        raise ValueError(f"positions must be [{plan.n_axes}, {tokens}], got {tuple(positions.shape)}")
    if tokens > 1 and positions.stride(-1) != 1:
        raise ValueError("positions must be contiguous along the tokens")
    return positions.data_ptr(), (positions.stride(0) if plan.n_axes > 1 else tokens)


def _overlap(a, b):
    """Whether two [T, heads, d] tensors share memory."""
    if a.numel() == 0 or b.numel() == 0 or a.untyped_storage().data_ptr() != b.untyped_storage().data_ptr():
        return False
    spans = []
    for t in (a, b):
        size = t.element_size()
        row, step = t.shape[1] * t.shape[2] * size, (t.stride(0) if t.shape[0] > 1 else 0) * size
        spans.append((t.data_ptr(), t.data_ptr() + (t.shape[0] - 1) * step + row, row, step))
    (a0, a1, ra, sa), (b0, b1, rb, sb) = spans
    if a1 <= b0 or b1 <= a0:
        return False
    if sa == sb and sa > 0:     # columns of the same rows: apart when their offsets within a row are
        d = (b0 - a0) % sa
        return d < ra or d + rb > sa
    return True


def _same(a, b):
    return a.data_ptr() == b.data_ptr() and a.shape == b.shape and a.stride() == b.stride()


def _check_outputs(outs, inputs):
    """An output may be the input beside it, and shares no memory otherwise."""
    if len(outs) > 1 and outs[0] is not None and outs[1] is not None and _overlap(*outs):
        raise ValueError("q_out and k_out overlap")
    for i, o in enumerate(outs):
        for j, t in enumerate(inputs):
            if o is not None and t is not None and not (i == j and _same(o, t)) and _overlap(o, t):
                raise ValueError("an output overlaps an input without being it")


def _rope(name, q, k, positions, plan, q_out, k_out, stream):
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q and k must be [T, heads, d]")
    dtype, dev = q.dtype, q.device
    if dtype is not _BF16 and dtype is not torch.float32:
        raise TypeError(f"unsupported dtype {dtype}")
    tokens, nq, hd = q.shape
    if hd != plan.head_dim:
        raise ValueError(f"the plan is for head_dim {plan.head_dim}, q has {hd}")
    qs = _rows(q, "q", tokens, nq, hd, dtype, dev)
    nk = kp = ks = kop = 0
    if k is not None:
        nk = k.shape[1]
        ks = _rows(k, "k", tokens, nk, hd, dtype, dev)
    elif k_out is not None:
        raise ValueError("k_out without k")
    pos, pos_stride = _positions(positions, plan, tokens, dev)
    qos, kos = nq * hd, nk * hd
    if q_out is not None or k_out is not None:
        if q_out is not None:
            qos = _rows(q_out, "q_out", tokens, nq, hd, dtype, dev)
        if k_out is not None:
            kos = _rows(k_out, "k_out", tokens, nk, hd, dtype, dev)
        _check_outputs((q_out, k_out), (q, k))
    index = q.get_device()
    if q_out is None:
        q_out = _empty(q, (tokens, nq, hd), dtype, stream)
    if k is not None and k_out is None:
        k_out = _empty(q, (tokens, nk, hd), dtype, stream)
    if tokens == 0:
        return q_out, k_out
    if k is not None:
        kp, kop = k.data_ptr(), k_out.data_ptr()
    _call(name, index, stream, plan.ref, q.data_ptr(), qs, kp, ks, pos, pos_stride, tokens, nq, nk,
          _lib.ZL_BF16 if dtype is _BF16 else _lib.ZL_FP32, q_out.data_ptr(), qos, kop, kos)
    return q_out, k_out


def rope_fwd(q, k, positions, plan, q_out=None, k_out=None, stream=None):
    """Turns q [T, Hq, d] and k [T, Hk, d] (or None) by their tokens' positions
    (int32 [T], or [n_axes, T]).  Returns (q_out, k_out); an output may be its
    own input."""
    if stream is None and q_out is None and k_out is None:
        r = _short("rope", False, q, k, positions, plan.address, plan.n_axes, plan.head_dim)
        if r is not None:
            return r
    return _rope("zl_rope_fwd", q, k, positions, plan, q_out, k_out, stream)


def rope_bwd(dq, dk, positions, plan, dq_out=None, dk_out=None, stream=None):
    """Gradient of rope_fwd: from the gradients of its outputs to those of its
    inputs.  Returns (dq_out, dk_out)."""
    if stream is None and dq_out is None and dk_out is None:
        r = _short("rope", True, dq, dk, positions, plan.address, plan.n_axes, plan.head_dim)
        if r is not None:
            return r
    return _rope("zl_rope_bwd", dq, dk, positions, plan, dq_out, dk_out, stream)


# ------------------------------------------------------------------ the cache
def _cache(k_pages, v_pages, page_table, kv_lens, seqs):
    """The checked zl_paged_cache_t, its key heads and head_dim."""
    if k_pages.dim() != 4 or page_table.dim() != 2:
        raise ValueError("k_pages must be [P, Hk, page, d] and page_table [S, cols]")
    dev, shape = k_pages.device, k_pages.shape
    if k_pages.dtype is not _BF16:
        raise TypeError("the pages must be bf16")
    cols = page_table.shape[1]
    if page_table.shape[0] != seqs:
        raise ValueError(f"page_table has {page_table.shape[0]} rows, the batch {seqs} sequences")
    if not k_pages.is_contiguous():
        raise ValueError("k_pages must be contiguous")
    _exact(v_pages, "v_pages", shape, _BF16, dev)
    _exact(page_table, "page_table", (seqs, cols), _I32, dev)
    _exact(kv_lens, "kv_lens", (seqs,), _I32, dev)
    p, nk, page, hd = shape
    return _CACHE.pack(k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), kv_lens.data_ptr(), cols, p,
                       page, nk, hd, 0), nk, hd


def paged_append(k, v, k_pages, v_pages, page_table, kv_lens, cu_seqlens, q=None, q_out=None, rope=None,
                 positions=None, stream=None, status=None):
    """Writes a batch's new tokens k, v [T, Hk, d] into the pages: sequence s's
    rows of cu_seqlens become its last positions below kv_lens[s].  With a
    RopePlan the keys (and q [T, H, d], if given) are turned at their cache
    positions, or at `positions`.  Returns the turned q (or None).

    kv_lens has to count the new tokens, and the pages they go to must be the
    sequence's own, as pages_extend sees to.  Where it reported anything but 0
    the lengths are the old ones, and the tokens would be written over the last
    ones of each sequence: unless the host has read 0 from it, give the tensor
    that it returned as `status`.  Then nothing is written unless it holds 0,
    and the next sync_check raises."""
    cu = _cu(cu_seqlens)
    if stream is None and q_out is None and positions is None:
        plan = 0 if rope is None else rope.address
        if status is None:
            r = _short("append", k, v, k_pages, v_pages, page_table, kv_lens, cu.address, cu.n, cu.last, q, plan)
        else:
            r = _short("append_after", k, v, k_pages, v_pages, page_table, kv_lens, cu.address, cu.n, cu.last, q, plan,
                       status)
        if r is not None:
            return r[0]
    cache, nk, hd = _cache(k_pages, v_pages, page_table, kv_lens, cu.n - 1)
    tokens, dev = cu.last, k_pages.device
    ks = _rows(k, "k", tokens, nk, hd, _BF16, dev)
    vs = _rows(v, "v", tokens, nk, hd, _BF16, dev)
    nq = qp = qs = qop = qos = pos = pos_stride = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError("q must be [T, H, d]")
        nq = q.shape[1]
        qs = _rows(q, "q", tokens, nq, hd, _BF16, dev)
        if q_out is None:
            q_out = _empty(q, (tokens, nq, hd), _BF16, stream)
            qos = nq * hd
        else:
            qos = _rows(q_out, "q_out", tokens, nq, hd, _BF16, dev)
            _check_outputs((q_out,), (q, k, v))
        qp, qop = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    if positions is not None:
        if rope is None:
            raise ValueError("positions without a rope plan")
        pos, pos_stride = _positions(positions, rope, tokens, dev)
    if status is not None:
        _exact(status, "status", (1,), _I32, dev)
    index = k_pages.get_device()
    if tokens == 0 and index >= 0:
        return q_out
    _call("zl_paged_append_ex", index, stream, cache, k.data_ptr(), ks, v.data_ptr(), vs, cu.array, cu.n - 1,
          None if rope is None else rope.ref, pos, pos_stride, qp, qs, nq, qop, qos,
          None if status is None else status.data_ptr())
    return q_out


def paged_attn_workspace_bytes(cu_seqlens_q, max_kv_len, num_heads, num_kv_heads, head_dim) -> int:
    lib = _lib.load()
    cu = _cu(cu_seqlens_q)
    for value, name in ((max_kv_len, "max_kv_len"), (num_heads, "num_heads"), (num_kv_heads, "num_kv_heads"),
                        (head_dim, "head_dim")):
        _int32(value, name)
    out = ctypes.c_size_t(0)
    _lib.check(lib.zl_paged_attn_workspace_size(cu.array, cu.n - 1, max_kv_len, num_heads, num_kv_heads, head_dim,
                                                ctypes.byref(out)), "zl_paged_attn_workspace_size")
    return int(out.value)


def paged_attn(q, k_pages, v_pages, page_table, kv_lens, cu_seqlens_q, max_kv_len, causal=True, window=0,
               softmax_scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of each sequence's new queries q [Tq, H, d] over its cached
    keys and values.  The queries stand at the last positions below kv_lens;
    max_kv_len (host) bounds kv_lens.  Returns (o [Tq, H, d], lse [H, Tq]).

    The same batch gives the same bits on every run; another batch around a
    sequence, or another bound, may change its last ones.  Behind a refused
    pages_extend the queries are taken for the last cached tokens: nothing is
    written to the cache, and the results mean nothing."""
    cu = _cu(cu_seqlens_q)
    if stream is None:
        r = _short("attn", q, k_pages, v_pages, page_table, kv_lens, cu.address, cu.n, cu.last, max_kv_len, causal,
                   window, softmax_scale, out, lse, workspace)
        if r is not None:
            return r
    _int32(max_kv_len, "max_kv_len")
    _int32(window, "window")
    cache, nk, hd = _cache(k_pages, v_pages, page_table, kv_lens, cu.n - 1)
    if q.dim() != 3:
        raise ValueError("q must be [Tq, H, d]")
    tq, nh, _ = q.shape
    if tq != cu.last:
        raise ValueError(f"q has {tq} rows, cu_seqlens_q ends at {cu.last}")
    dev = k_pages.device
    qs = _rows(q, "q", tq, nh, hd, _BF16, dev)
    if out is not None:
        _exact(out, "out", (tq, nh, hd), _BF16, dev)
    if lse is not None:
        _exact(lse, "lse", (nh, tq), torch.float32, dev)
    index = q.get_device()
    if index < 0:
        raise ValueError("tensors must be CUDA tensors")
    if out is None:
        out = _empty(q, (tq, nh, hd), _BF16, stream)
    if lse is None:
        lse = _empty(q, (nh, tq), torch.float32, stream)
    if workspace is None:
        workspace = _empty(q, (paged_attn_workspace_bytes(cu, max_kv_len, nh, nk, hd),), torch.uint8, stream)
    ws, ws_bytes = _scratch(workspace, dev)
    _call("zl_paged_attn", index, stream, cache, q.data_ptr(), qs, cu.array, cu.n - 1, max_kv_len, nh,
          1.0 / math.sqrt(hd) if softmax_scale is None else softmax_scale, 1 if causal else 0, window, out.data_ptr(),
          lse.data_ptr(), ws, ws_bytes)
    return out, lse


# ------------------------------------------------------------------ whole pages
def _tables(page_table, kv_lens, page_refs, page_size):
    """The checked zl_page_tables_t, and the device."""
    if page_table.dim() != 2 or page_refs.dim() != 1:
        raise ValueError("page_table must be [S, cols] and page_refs [P]")
    _int32(page_size, "page_size")
    dev = page_table.device
    slots, cols = page_table.shape
    pages = page_refs.shape[0]
    for value, name in ((slots, "the table's rows"), (cols, "the table's columns"), (pages, "the number of pages")):
        _int32(value, name)
    _exact(page_table, "page_table", (slots, cols), _I32, dev)
    _exact(kv_lens, "kv_lens", (slots,), _I32, dev)
    _exact(page_refs, "page_refs", (pages,), _I32, dev)
    return _TABLES.pack(page_table.data_ptr(), kv_lens.data_ptr(), page_refs.data_ptr(), slots, cols, pages,
                        page_size), dev


def _pool(cache, num_pages=None, device=None):
    """The checked zl_page_pool_t of cache [..., P, Hk, page, d]; the dimensions
    before P (layers, keys and values) are the groups."""
    shape = cache.shape
    if len(shape) < 4:
        raise ValueError("the cache must be [..., P, Hk, page, d]")
    p = shape[-4]
    if num_pages is not None and p != num_pages:
        raise ValueError(f"the cache has {p} pages, page_refs {num_pages}")
    if device is not None and cache.device != device:
        raise ValueError(f"the cache must be on {device}")
    if not cache.is_contiguous():
        raise ValueError("the cache must be contiguous")
    page = shape[-3] * shape[-2] * shape[-1]
    size = page * cache.element_size()
    return _POOL.pack(cache.data_ptr(), size, p * size, cache.numel() // max(1, p * page), p)


def _list(t, name, device):
    if t.dim() != 1:
        raise ValueError(f"{name} must be a vector")
    _int32(t.shape[0], f"the length of {name}")
    _exact(t, name, t.shape, _I32, device)
    return t.shape[0]


def _status(status, like, stream):
    if status is None:
        return _empty(like, (1,), _I32, stream)
    _exact(status, "status", (1,), _I32, like.device)
    return status


def _pages_scratch(workspace, like, num_pages, stream):
    if workspace is None:
        workspace = _empty(like, (pages_workspace_bytes(num_pages),), torch.uint8, stream)
    ws, size = _scratch(workspace, like.device)
    return workspace, ws, size


def pages_workspace_bytes(num_pages) -> int:
    _int32(num_pages, "num_pages")
    out = ctypes.c_size_t(0)
    _lib.check(_lib.load().zl_pages_workspace_size(num_pages, ctypes.byref(out)), "zl_pages_workspace_size")
    return int(out.value)


def pages_extend(page_table, kv_lens, page_refs, counts, page_size, status=None, stream=None):
    """Makes room for counts[s] (int32, device) new tokens in every slot, in
    place: kv_lens grows, free pages (lowest first) enter the rows.  Returns a
    device int32 [1]: 0, or the pages lacking, or -1 for counts that are
    negative or do not fit a row, or -2 for a slot that would grow inside a page
    that another one holds (it was truncated there); unless it is 0 nothing was
    changed."""
    if stream is None and status is None:
        r = _short("extend", page_table, kv_lens, page_refs, counts, page_size)
        if r is not None:
            return r
    t, dev = _tables(page_table, kv_lens, page_refs, page_size)
    _exact(counts, "counts", kv_lens.shape, _I32, dev)
    status = _status(status, kv_lens, stream)
    _call("zl_pages_extend", kv_lens.get_device(), stream, t, counts.data_ptr(), status.data_ptr())
    return status


def pages_fork(cache, page_table, kv_lens, page_refs, parents, children, status=None, workspace=None, stream=None):
    """Makes each empty slot children[i] a copy of slot parents[i] (int32,
    device), in place: full pages are shared, a part-filled last page is copied
    in every group of cache [..., P, Hk, page, d].  Returns a device int32 [1]
    as pages_extend does."""
    if stream is None and status is None and workspace is not None:
        r = _short("fork", cache, page_table, kv_lens, page_refs, parents, children, workspace)
        if r is not None:
            return r
    t, dev = _tables(page_table, kv_lens, page_refs, cache.shape[-2] if cache.dim() >= 2 else 0)
    p = _pool(cache, page_refs.shape[0], dev)
    n = _list(parents, "parents", dev)
    if _list(children, "children", dev) != n:
        raise ValueError("parents and children differ in length")
    status = _status(status, kv_lens, stream)
    workspace, ws, size = _pages_scratch(workspace, kv_lens, page_refs.shape[0], stream)
    _call("zl_pages_fork", kv_lens.get_device(), stream, p, t, parents.data_ptr(), children.data_ptr(), n,
          status.data_ptr(), ws, size)
    return status


def pages_free(page_table, kv_lens, page_refs, slots, page_size, stream=None):
    """Empties the slots (int32, device), in place."""
    t, dev = _tables(page_table, kv_lens, page_refs, page_size)
    n = _list(slots, "slots", dev)
    _call("zl_pages_free", kv_lens.get_device(), stream, t, slots.data_ptr(), n)


def pages_truncate(page_table, kv_lens, page_refs, lens, page_size, stream=None):
    """Shortens every slot that is longer than lens[s] (int32, device) to it, in
    place, as when drafted tokens are taken back; the pages behind are freed.
    A slot cut inside a page that another one holds (a fork's parent or child,
    shortened to before the fork) cannot be extended until it has that page to
    itself: fork it to an empty slot and free it."""
    t, dev = _tables(page_table, kv_lens, page_refs, page_size)
    _exact(lens, "lens", kv_lens.shape, _I32, dev)
    _call("zl_pages_truncate", kv_lens.get_device(), stream, t, lens.data_ptr())


def pages_compact(cache, page_table, kv_lens, page_refs, live=None, workspace=None, stream=None):
    """Moves the used pages to the front of the pool, in place, in every group
    of cache [..., P, Hk, page, d].  Returns their number, a device int32 [1]."""
    if stream is None and live is None and workspace is not None:
        r = _short("compact", cache, page_table, kv_lens, page_refs, workspace)
        if r is not None:
            return r
    t, dev = _tables(page_table, kv_lens, page_refs, cache.shape[-2] if cache.dim() >= 2 else 0)
    p = _pool(cache, page_refs.shape[0], dev)
    live = _status(live, kv_lens, stream)
    workspace, ws, size = _pages_scratch(workspace, kv_lens, page_refs.shape[0], stream)
    _call("zl_pages_compact", kv_lens.get_device(), stream, p, t, live.data_ptr(), ws, size)
    return live


def pages_copy(cache, src, dst, stream=None):
    """Copies page src[i] over page dst[i] (int32, device) in every group of
    cache [..., P, Hk, page, d]; no page may be both, nor a target twice."""
    p = _pool(cache)
    n = _list(src, "src", cache.device)
    if _list(dst, "dst", cache.device) != n:
        raise ValueError("src and dst differ in length")
    _call("zl_pages_copy", cache.get_device(), stream, p, src.data_ptr(), dst.data_ptr(), n)
