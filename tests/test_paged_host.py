"""Host checks of rotary positions and the paged cache, without a GPU: plans,
refusals of the C ABI and of the binding, and the oracle's own facts."""
import copy
import ctypes
import gc
import math
import pickle

import numpy as np
import pytest
import torch

import mixed_length_dit_gb300 as zl
from mixed_length_dit_gb300 import _lib
from oracle import paged_f64 as ref

P64 = ctypes.c_void_p(64)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


# ------------------------------------------------------------------ plans
@pytest.mark.parametrize("kw", [
    {}, {"axes": (64,)}, {"axes": (44, 42, 42), "interleaved": True}, {"base": 500000.0, "factor": 8.0},
    {"factor": 4.0, "ramp": (1.0, 4.0, 8192)}, {"axes": (2,), "magnitude": 1.25},
])
def test_plan_steps_are_the_frequencies(kw):
    plan = zl.RopePlan(128, **kw)
    axes = kw.get("axes", (128,))
    freq, axis = ref.rope_frequencies(axes, kw.get("base", 10000.0), kw.get("factor", 1.0), kw.get("ramp"))
    step = np.array([plan.struct.step[i] for i in range(len(freq))], dtype=np.float64) / 2.0 ** 64
    # a relative 4 * 2^-53 of the frequency, plus the fraction's last bit
    assert np.all(np.abs(step - freq / (2 * math.pi)) <= 2.0 ** -50 * freq + 2.0 ** -63)
    ends = [plan.struct.pair_end[a] for a in range(len(axes))]
    assert ends == list(np.cumsum([d // 2 for d in axes]))
    assert plan.struct.rot_dim == sum(axes) and plan.struct.interleaved == int(kw.get("interleaved", False))


@pytest.mark.parametrize("args,kw,status", [
    ((96,), {}, _lib.ZL_EUNSUPPORTED),
    ((64,), {"axes": (66,)}, _lib.ZL_EINVAL),
    ((64,), {"axes": (3,)}, _lib.ZL_EINVAL),
    ((64,), {"axes": (0, 4)}, _lib.ZL_EINVAL),
    ((64,), {"axes": ()}, _lib.ZL_EINVAL),
    ((64,), {"axes": (4, 4, 4, 4, 4)}, _lib.ZL_EINVAL),
    ((64,), {"base": 1.0}, _lib.ZL_EINVAL),
    ((64,), {"base": float("nan")}, _lib.ZL_EINVAL),
    ((64,), {"factor": 0.0}, _lib.ZL_EINVAL),
    ((64,), {"magnitude": 0.0}, _lib.ZL_EINVAL),
    ((64,), {"magnitude": 1e300}, _lib.ZL_EINVAL),
    ((64,), {"ramp": (4.0, 1.0, 100)}, _lib.ZL_EINVAL),
    ((64,), {"ramp": (1.0, 4.0, 0)}, _lib.ZL_EINVAL),
])
def test_plan_refusals(args, kw, status):
    with pytest.raises(zl.ZlError) as e:
        zl.RopePlan(*args, **kw)
    assert e.value.status == status


# ------------------------------------------------------------------ the C ABI
def _rope_call(lib, fn="zl_rope_fwd", plan=None, q=64, qs=128, k=64, ks=64, pos=64, ps=10, t=10, nq=2, nk=1,
               dtype=_lib.ZL_BF16, qo=64, ko=64):
    plan = zl.RopePlan(64).struct if plan is None else plan
    return getattr(lib, fn)(ctypes.byref(plan), q, qs, k, ks, pos, ps, t, nq, nk, dtype, qo, qs, ko, ks, None)


@pytest.mark.parametrize("fn", ["zl_rope_fwd", "zl_rope_bwd"])
def test_rope_refusals(lib, fn):
    assert _rope_call(lib, fn, t=0) == _lib.ZL_OK
    assert _rope_call(lib, fn, dtype=5) == _lib.ZL_EUNSUPPORTED
    assert _rope_call(lib, fn, t=-1) == _lib.ZL_EINVAL
    assert _rope_call(lib, fn, nq=0) == _lib.ZL_EINVAL
    assert _rope_call(lib, fn, q=0) == _lib.ZL_EINVAL
    assert _rope_call(lib, fn, pos=0) == _lib.ZL_EINVAL
    assert _rope_call(lib, fn, pos=66) == _lib.ZL_EALIGN
    assert _rope_call(lib, fn, qs=64) == _lib.ZL_EINVAL             # heads do not fit the row
    assert _rope_call(lib, fn, qs=129) == _lib.ZL_EALIGN
    assert _rope_call(lib, fn, k=8) == _lib.ZL_EALIGN
    assert _rope_call(lib, fn, ko=0) == _lib.ZL_EINVAL
    bad = zl.RopePlan(64).struct
    bad.rot_dim = 63
    assert _rope_call(lib, fn, plan=bad) == _lib.ZL_EINVAL
    bad = zl.RopePlan(64, axes=(32, 32)).struct
    assert _rope_call(lib, fn, plan=bad, ps=9) == _lib.ZL_EINVAL    # the axes' rows overlap
    bad.pair_end[0] = 40
    assert _rope_call(lib, fn, plan=bad) == _lib.ZL_EINVAL


def _cache(**kw):
    f = dict(k_pages=64, v_pages=64, page_table=64, kv_lens=64, table_cols=8, num_pages=20, page_size=16,
             num_kv_heads=2, head_dim=64, reserved=0)
    f.update(kw)
    return _lib.PagedCache(*f.values())


CACHE_FAULTS = [
    (dict(head_dim=80), _lib.ZL_EUNSUPPORTED), (dict(page_size=48), _lib.ZL_EUNSUPPORTED),
    (dict(page_size=8), _lib.ZL_EUNSUPPORTED), (dict(page_size=512), _lib.ZL_EUNSUPPORTED),
    (dict(table_cols=0), _lib.ZL_EINVAL), (dict(num_pages=0), _lib.ZL_EINVAL),
    (dict(num_kv_heads=0), _lib.ZL_EINVAL), (dict(num_pages=1 << 28), _lib.ZL_EINVAL),
    (dict(table_cols=1 << 28), _lib.ZL_EINVAL), (dict(reserved=1), _lib.ZL_EINVAL),
    (dict(k_pages=0), _lib.ZL_EINVAL), (dict(v_pages=8), _lib.ZL_EALIGN), (dict(kv_lens=66), _lib.ZL_EALIGN),
    (dict(page_table=0), _lib.ZL_EINVAL),
]


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_append_and_attn_refuse_bad_caches(lib, fault, status):
    cu, n = _lib.int32_array([0, 3])
    c = _cache(**fault)
    assert lib.zl_paged_append(ctypes.byref(c), P64, 128, P64, 128, cu, n - 1, None, None, 0, None, 0, 0, None, 0,
                               None) == status
    nk = fault.get("num_kv_heads", 2) or 1
    assert lib.zl_paged_attn(ctypes.byref(c), P64, 4 * nk * 64, cu, n - 1, 100, 4 * nk, 0.125, 1, 0, P64, P64, P64,
                             1 << 40, None) == status


def test_append_refusals(lib):
    def call(cu=(0, 3), plan=None, pos=None, ps=0, q=None, qs=0, nq=0, qo=None, k=64, ks=128):
        arr, n = _lib.int32_array(cu)
        c = _cache()
        return lib.zl_paged_append(ctypes.byref(c), k, ks, P64, 128, arr, n - 1,
                                   None if plan is None else ctypes.byref(plan.struct), pos, ps, q, qs, nq, qo, qs, None)
    assert call(cu=(0,)) == _lib.ZL_OK
    assert call(cu=(0, 0, 0)) == _lib.ZL_OK
    assert call(cu=(1, 3)) == _lib.ZL_EINVAL
    assert call(cu=(0, 3, 2)) == _lib.ZL_EINVAL
    assert call(plan=zl.RopePlan(128)) == _lib.ZL_EINVAL            # another head_dim
    assert call(plan=zl.RopePlan(64, axes=(32, 32))) == _lib.ZL_EINVAL   # two axes need positions
    assert call(pos=64) == _lib.ZL_EINVAL                           # positions without a plan
    assert call(q=64, qs=128) == _lib.ZL_EINVAL                     # q without heads
    assert call(nq=2) == _lib.ZL_EINVAL                             # heads without q
    assert call(q=64, qs=128, nq=2, qo=None) == _lib.ZL_EINVAL
    assert call(k=None) == _lib.ZL_EINVAL
    assert call(ks=120) == _lib.ZL_EINVAL


def test_attn_refusals(lib):
    def call(cu=(0, 3), q=64, qs=256, most=100, nh=4, scale=0.125, causal=1, window=0, o=64, lse=64):
        arr, n = _lib.int32_array(cu)
        c = _cache()
        return lib.zl_paged_attn(ctypes.byref(c), q, qs, arr, n - 1, most, nh, scale, causal, window, o, lse, P64,
                                 1 << 40, None)
    assert call(cu=(0, 0), q=None, o=None) == _lib.ZL_OK
    assert call(cu=(0, 3, 1)) == _lib.ZL_EINVAL
    assert call(nh=3) == _lib.ZL_EINVAL                             # not a multiple of the key heads
    assert call(nh=2 * 129, qs=2 * 129 * 64) == _lib.ZL_EUNSUPPORTED
    assert call(most=-1) == _lib.ZL_EINVAL
    assert call(most=8 * 16 + 1) == _lib.ZL_EINVAL                  # longer than a table row
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert call(scale=scale) == _lib.ZL_EINVAL
    assert call(causal=2) == _lib.ZL_EINVAL
    assert call(window=-1) == _lib.ZL_EINVAL
    assert call(q=None) == _lib.ZL_EINVAL
    assert call(qs=200) == _lib.ZL_EINVAL
    assert call(qs=258) == _lib.ZL_EALIGN
    assert call(o=8) == _lib.ZL_EALIGN
    assert call(lse=None) == _lib.ZL_EINVAL


def test_attn_workspace_rules(lib):
    out = ctypes.c_size_t(0)

    def size(cu, most, nh, nk, hd):
        arr, n = _lib.int32_array(cu)
        return lib.zl_paged_attn_workspace_size(arr, n - 1, most, nh, nk, hd, ctypes.byref(out))
    assert size((0, 3), 100, 4, 2, 64) == _lib.ZL_OK
    assert size((0, 3), 100, 4, 3, 64) == _lib.ZL_EINVAL
    assert size((0, 3), 100, 4, 2, 96) == _lib.ZL_EUNSUPPORTED
    assert size((0, 3), -5, 4, 2, 64) == _lib.ZL_EINVAL
    assert size((0,), 0, 4, 2, 64) == _lib.ZL_OK and out.value == 0


def _tables(**kw):
    f = dict(page_table=64, kv_lens=64, page_refs=64, slots=4, table_cols=8, num_pages=20, page_size=16)
    f.update(kw)
    return _lib.PageTables(*f.values())


def _pool(**kw):
    f = dict(base=64, page_bytes=4096, group_stride=20 * 4096, groups=2, num_pages=20)
    f.update(kw)
    return _lib.PagePool(*f.values())


@pytest.mark.parametrize("fault,status", [
    (dict(page_size=24), _lib.ZL_EUNSUPPORTED), (dict(slots=0), _lib.ZL_EINVAL), (dict(slots=8193), _lib.ZL_EINVAL),
    (dict(table_cols=0), _lib.ZL_EINVAL), (dict(num_pages=0), _lib.ZL_EINVAL), (dict(page_refs=0), _lib.ZL_EINVAL),
    (dict(kv_lens=65), _lib.ZL_EALIGN), (dict(table_cols=1 << 28), _lib.ZL_EINVAL),
])
def test_page_tables_refusals(lib, fault, status):
    t, p = _tables(**fault), _pool(num_pages=fault.get("num_pages", 20) or 20)
    assert lib.zl_pages_extend(ctypes.byref(t), P64, P64, None) == status
    assert lib.zl_pages_free(ctypes.byref(t), P64, 1, None) == status
    assert lib.zl_pages_fork(ctypes.byref(p), ctypes.byref(t), P64, P64, 1, P64, P64, 1 << 30, None) == status
    assert lib.zl_pages_compact(ctypes.byref(p), ctypes.byref(t), P64, P64, 1 << 30, None) == status


@pytest.mark.parametrize("fault,status", [
    (dict(base=0), _lib.ZL_EINVAL), (dict(base=72), _lib.ZL_EALIGN), (dict(page_bytes=0), _lib.ZL_EINVAL),
    (dict(page_bytes=24), _lib.ZL_EINVAL), (dict(groups=0), _lib.ZL_EINVAL), (dict(num_pages=0), _lib.ZL_EINVAL),
    (dict(group_stride=4096), _lib.ZL_EINVAL), (dict(page_bytes=1 << 40), _lib.ZL_EINVAL),
])
def test_page_pool_refusals(lib, fault, status):
    t, p = _tables(), _pool(**fault)
    assert lib.zl_pages_copy(ctypes.byref(p), P64, P64, 3, None) == status
    assert lib.zl_pages_fork(ctypes.byref(p), ctypes.byref(t), P64, P64, 1, P64, P64, 1 << 30, None) == status


def test_page_operation_arguments(lib):
    t, p = _tables(), _pool()
    tp, pp = ctypes.byref(t), ctypes.byref(p)
    assert lib.zl_pages_extend(tp, None, P64, None) == _lib.ZL_EINVAL
    assert lib.zl_pages_free(tp, None, 0, None) == _lib.ZL_OK
    assert lib.zl_pages_free(tp, None, 2, None) == _lib.ZL_EINVAL
    assert lib.zl_pages_fork(pp, tp, P64, P64, -1, P64, P64, 1 << 30, None) == _lib.ZL_EINVAL
    assert lib.zl_pages_fork(pp, tp, P64, P64, 2, P64, P64, 16, None) == _lib.ZL_EWORKSPACE
    assert lib.zl_pages_compact(pp, tp, P64, None, 1 << 30, None) == _lib.ZL_EWORKSPACE
    assert lib.zl_pages_compact(pp, tp, None, P64, 1 << 30, None) == _lib.ZL_EINVAL
    other = _pool(num_pages=19)
    assert lib.zl_pages_compact(ctypes.byref(other), tp, P64, P64, 1 << 30, None) == _lib.ZL_EINVAL
    assert lib.zl_pages_copy(pp, None, None, 0, None) == _lib.ZL_OK
    out = ctypes.c_size_t(0)
    assert lib.zl_pages_workspace_size(20, ctypes.byref(out)) == _lib.ZL_OK and out.value >= 3 * 20 * 4
    assert lib.zl_pages_workspace_size(0, ctypes.byref(out)) == _lib.ZL_EINVAL


# ------------------------------------------------------------------ the binding
def _b(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_rope_binding_refusals():
    plan = zl.RopePlan(64)
    q, k, pos = _b(5, 4, 64), _b(5, 2, 64), _i(5)
    for args, match in [
        ((_b(5, 256), k, pos, plan), "must be"), ((_b(5, 4, 128), None, pos, plan), "head_dim"),
        ((q, _b(4, 2, 64), pos, plan), "k must be"), ((q, _b(5, 2, 64, dtype=torch.float32), pos, plan), "k must be"),
        ((q, k, _i(4), plan), "positions"), ((q, k, pos.long(), plan), "positions"),
        ((q, k, _i(2, 5), plan), "positions"), ((q, k, pos, zl.RopePlan(64, axes=(32, 32))), "positions"),
        ((_b(4, 5, 64).transpose(0, 1), k, pos, plan), "contiguous"),
    ]:
        with pytest.raises(ValueError, match=match):
            zl.rope_fwd(*args)
    with pytest.raises(TypeError):
        zl.rope_fwd(q.half(), None, pos, plan)
    rows = _b(6, 4, 64)
    with pytest.raises(ValueError, match="overlaps"):
        zl.rope_fwd(rows[:5], None, pos, plan, q_out=rows[1:])
    fused = _b(5, 8, 64)
    with pytest.raises(ValueError, match="overlap"):
        zl.rope_fwd(fused[:, :4], fused[:, 4:6], pos, plan, q_out=fused[:, 2:6])
    with pytest.raises(ValueError, match="q_out and k_out"):
        zl.rope_fwd(q, q, pos, plan, q_out=q, k_out=q)
    with pytest.raises(ValueError, match="CUDA"):      # parts of one row: no overlap, but not on the GPU
        zl.rope_fwd(fused[:, :4], fused[:, 4:6], pos, plan, q_out=fused[:, :4], k_out=fused[:, 4:6])


def test_paged_binding_refusals():
    kp, vp, table, lens = _b(10, 2, 16, 64), _b(10, 2, 16, 64), _i(2, 4), _i(2)
    k, q, cu = _b(5, 2, 64), _b(5, 4, 64), [0, 2, 5]
    with pytest.raises(ValueError, match="page_table has"):
        zl.paged_append(k, k, kp, vp, table, lens, [0, 5])
    with pytest.raises(ValueError, match="k must be"):
        zl.paged_append(_b(4, 2, 64), k, kp, vp, table, lens, cu)
    with pytest.raises(ValueError, match="v_pages must be"):
        zl.paged_append(k, k, kp, vp[:9], table, lens, cu)
    with pytest.raises(ValueError, match="kv_lens must be"):
        zl.paged_append(k, k, kp, vp, table, lens.long(), cu)
    with pytest.raises(ValueError, match="positions without"):
        zl.paged_append(k, k, kp, vp, table, lens, cu, positions=_i(5))
    with pytest.raises(ValueError, match="q_out without"):
        zl.paged_append(k, k, kp, vp, table, lens, cu, q_out=q)
    with pytest.raises(ValueError, match="CUDA"):
        zl.paged_append(k, k, kp, vp, table, lens, cu)
    with pytest.raises(ValueError, match="q has 4 rows"):
        zl.paged_attn(q[:4], kp, vp, table, lens, cu, 40)
    with pytest.raises(ValueError, match="q must be"):
        zl.paged_attn(_b(5, 4, 128), kp, vp, table, lens, cu, 40)
    with pytest.raises(ValueError, match="lse must be"):
        zl.paged_attn(q, kp, vp, table, lens, cu, 40, lse=_b(5, 4, dtype=torch.float32))
    with pytest.raises(TypeError):
        zl.paged_attn(q, kp.float(), vp.float(), table, lens, cu, 40)
    with pytest.raises(ValueError, match="CUDA"):
        zl.paged_attn(q, kp, vp, table, lens, cu, 40)
    with pytest.raises(ValueError, match="contiguous"):
        zl.paged_attn(q, kp.transpose(1, 2).contiguous().transpose(1, 2), vp, table, lens, cu, 40)


def test_pages_binding_refusals():
    cache, table, lens, refs = _b(3, 10, 2, 16, 64), _i(2, 4), _i(2), _i(10)
    with pytest.raises(ValueError, match="counts must be|CUDA"):
        zl.pages_extend(table, lens, refs, _i(3), 16)
    with pytest.raises(ValueError, match="page_refs"):
        zl.pages_extend(table, lens, _i(10, 1), _i(2), 16)
    with pytest.raises(ValueError, match="CUDA"):
        zl.pages_fork(cache, table, lens, refs, _i(1), _i(1))
    with pytest.raises(ValueError, match="CUDA"):
        zl.pages_copy(cache, _i(1), _i(1))
    with pytest.raises(ValueError, match=r"\[\.\.\., P"):
        zl.pages_copy(_b(10, 2), _i(1), _i(1))


def test_host_int32_is_taken_as_it_is():
    a = zl.host_int32([0, 3, 7])
    assert len(a) == 3 and a.last == 7 and list(a) == [0, 3, 7]
    assert _lib.int32_array(a)[0] is a.array
    with pytest.raises(ValueError, match="at least one"):
        zl.paged_attn_workspace_bytes([], 10, 4, 2, 64)


# ------------------------------------------------------------------ the oracle's facts
def test_oracle_rope_facts():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((7, 2, 64))
    pos = rng.integers(-50, 50, (2, 7))
    for il in (False, True):
        y = ref.rope(x, pos, (20, 32), interleaved=il)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
        assert np.array_equal(y[..., 52:], x[..., 52:])
        assert np.allclose(ref.rope(y, pos, (20, 32), interleaved=il, sign=-1), x)      # the transpose undoes it
        assert np.array_equal(ref.rope(x, 0 * pos, (20, 32), interleaved=il), x)
        # scores of turned queries and keys depend on distances alone
        a, b = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
        dot = [float((ref.rope(a, [[p + 9]], (64,), interleaved=il) * ref.rope(b, [[p]], (64,), interleaved=il)).sum())
               for p in (0, 5, 1000)]
        assert np.allclose(dot, dot[0])


def test_oracle_rope_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, g = rng.standard_normal((3, 1, 64)), rng.standard_normal((3, 1, 64))
    pos = np.array([[3, 70, 1000]])
    grad = ref.rope(g, pos, (48,), magnitude=1.5, sign=-1)
    for i in (0, 17, 30, 50):
        d = np.zeros_like(x)
        d[1, 0, i] = 1e-5
        num = (g * (ref.rope(x + d, pos, (48,), magnitude=1.5) - ref.rope(x - d, pos, (48,), magnitude=1.5))).sum() / 2e-5
        assert abs(num - grad[1, 0, i]) < 1e-8


def test_oracle_attention_facts():
    rng = np.random.default_rng(2)
    kp, vp = rng.standard_normal((2, 6, 2, 16, 64))
    table, lens, cu = [[4, 1, 3], [0, -1, -1]], [40, 3], [0, 2, 5]
    q = rng.standard_normal((5, 4, 64))
    o, lse, _ = ref.paged_attn(q, kp, vp, table, lens, cu)
    assert np.allclose(o[2], np.repeat(vp[0, :, 0], 2, axis=0))     # the first token sees itself alone
    full, _, _ = ref.paged_attn(q, kp, vp, table, lens, cu, causal=False)
    assert np.allclose(full[[1, 4]], o[[1, 4]])                     # the last query sees all either way
    one, _, _ = ref.paged_attn(q, kp, vp, table, lens, cu, window=1)
    assert np.allclose(one[1], np.repeat(vp[3, :, 39 - 32], 2, axis=0))
    none, l_none, _ = ref.paged_attn(q, kp, vp, table, [1, 0], cu)
    assert np.all(none[0] == 0) and np.isneginf(l_none[:, 0]).all() and np.isfinite(l_none[:, 1]).all()
    assert np.all(none[2:] == 0)


def test_oracle_pages_facts():
    p = ref.Pages([[2, 5, -1], [-1] * 3, [-1] * 3], [20, 0, 0], [0, 0, 1, 0, 0, 1], 16)
    assert p.fork([0, 0], [1, 2]) == 0
    assert p.table[1][:2] == [2, 0] and p.table[2][:2] == [2, 1] and p.refs == [1, 1, 3, 0, 0, 1]
    assert p.data[:2] == [5, 5]
    p.release([0])
    assert p.refs == [1, 1, 2, 0, 0, 0] and p.table[0] == [-1] * 3
    assert p.extend([50, 0, 0]) == -1 and p.extend([48, 13, 0]) == 1 and p.lens[0] == 0
    assert p.extend([33, 0, 0]) == 0 and p.table[0] == [3, 4, 5]
    p.release([1])
    assert p.compact() == 5 and p.table[0] == [3, 4, 0]


def test_numbers_past_32_bits_are_refused():
    # ctypes would keep their low bits: a window of 2**32 + 5 would be one of 5
    k, v, t, n = (torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16),
                  torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32))
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="window"):
        zl.paged_attn(q, k, v, t, n, [0, 1], 16, window=2**32 + 5)
    with pytest.raises(ValueError, match="max_kv_len"):
        zl.paged_attn(q, k, v, t, n, [0, 1], 2**32 + 16)
    with pytest.raises(ValueError, match="max_kv_len"):
        zl.paged_attn_workspace_bytes([0, 1], 2**32 + 16, 1, 1, 64)
    with pytest.raises(ValueError, match="page_size"):
        zl.pages_extend(t, n, torch.zeros(2, dtype=torch.int32), n, 2**32 + 16)
    with pytest.raises(ValueError, match="num_pages"):
        zl.pages_workspace_bytes(2**32 + 1)


def test_compiled_binding_leaves_unusual_calls_alone():
    """It does nothing with what is not as it should be: the long way says why."""
    b = zl._lib.bind()
    cpu = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    pages, i1, i2 = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16), torch.ones(1, dtype=torch.int32), torch.zeros(
        1, 2, dtype=torch.int32)
    plan, cu = zl.RopePlan(64), zl.host_int32([0, 1])
    good = {
        "rope": [False, cpu, None, i1, plan.address, 1, 64],
        "append": [cpu, cpu, pages, pages, i2, i1, cu.address, 2, 1, None, 0],
        "attn": [cpu, pages, pages, i2, i1, cu.address, 2, 1, 16, True, 0, None, None, None, None],
        "extend": [i2, i1, i1, i1, 16],
        "fork": [pages, i2, i1, torch.zeros(2, dtype=torch.int32), i1, i1, i1],
        "compact": [pages, i2, i1, torch.zeros(2, dtype=torch.int32), i1],
    }
    for name, args in good.items():
        fn = getattr(b, name)
        assert fn(*args) is None                  # tensors of the CPU
        assert fn() is None and fn(*args[:-1]) is None and fn(*args, 1) is None
        for i in range(len(args)):
            for bad in (None, "x", 2**80, 1.5, torch.zeros(0), [1]):
                assert fn(*args[:i], bad, *args[i + 1:]) is None


@pytest.mark.parametrize("fault,status", [
    (dict(page_size=24), _lib.ZL_EUNSUPPORTED), (dict(slots=0), _lib.ZL_EINVAL), (dict(page_refs=0), _lib.ZL_EINVAL),
    (dict(kv_lens=65), _lib.ZL_EALIGN), (dict(table_cols=1 << 28), _lib.ZL_EINVAL),
])
def test_truncate_refusals(lib, fault, status):
    assert lib.zl_pages_truncate(ctypes.byref(_tables(**fault)), P64, None) == status
    assert lib.zl_pages_truncate(None, P64, None) == _lib.ZL_EINVAL
    assert lib.zl_pages_truncate(ctypes.byref(_tables()), None, None) == _lib.ZL_EINVAL
    assert lib.zl_pages_truncate(ctypes.byref(_tables()), 66, None) == _lib.ZL_EALIGN
    with pytest.raises(ValueError, match="lens"):
        zl.pages_truncate(_i(3, 4), _i(3), _i(20), _i(2), 16)
    with pytest.raises(ValueError, match="CUDA"):
        zl.pages_truncate(_i(3, 4), _i(3), _i(20), _i(3), 16)


def test_oracle_pages_shared_ends():
    p = ref.Pages([[0, 1, 2], [-1] * 3], [40, 0], [1, 1, 1, 0, 0], 16)
    assert p.fork([0], [1]) == 0
    p.truncate([40, 20])
    assert p.refs[1] == 2 and p.extend([0, 1]) == -2 and p.lens == [40, 20] and p.extend([3, 0]) == 0
    p.truncate([43, 16])
    assert p.refs[1] == 1 and p.extend([0, 5]) == 0 and p.table[1][1] != p.table[0][1]


def test_append_with_a_status_refusals(lib):
    cu, n = _lib.int32_array([0, 3])
    c = _cache()

    def call(status, k=64):
        return lib.zl_paged_append_ex(ctypes.byref(c), k, 128, P64, 128, cu, n - 1, None, None, 0, None, 0, 0, None, 0,
                                      status, None)
    assert call(66) == _lib.ZL_EALIGN
    assert call(64, k=None) == _lib.ZL_EINVAL
    kp, table, lens, k = _b(10, 2, 16, 64), _i(2, 4), _i(2), _b(5, 2, 64)
    for status in (_i(2), _i(1, 1), _i(1).long()):
        with pytest.raises(ValueError, match="status must be"):
            zl.paged_append(k, k, kp, kp, table, lens, [0, 2, 5], status=status)
    with pytest.raises(ValueError, match="CUDA"):
        zl.paged_append(k, k, kp, kp, table, lens, [0, 2, 5], status=_i(1))
    plan, hcu = zl.RopePlan(64), zl.host_int32([0, 2, 5])
    args = [k, k, kp, kp, table, lens, hcu.address, 3, 5, None, plan.address, _i(1)]
    fn = zl._lib.bind().append_after
    assert fn(*args) is None and fn() is None and fn(*args[:-1]) is None and fn(*args, 1) is None
    for i in range(len(args)):
        for bad in (None, "x", 2**80, 1.5, torch.zeros(0), [1]):
            assert fn(*args[:i], bad, *args[i + 1:]) is None


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))])
def test_copies_of_plans_and_host_arrays_point_at_their_own_memory(how):
    """A model that holds them is copied and pickled with them."""
    a = zl.host_int32([0, 3, 7])
    plan = zl.RopePlan(128, axes=(44, 42, 42), interleaved=True, factor=4.0, magnitude=1.25)
    b, c = how(a), how(plan)
    assert b.address == ctypes.addressof(b.array) and list(b) == [0, 3, 7] and (b.n, b.last) == (3, 7)
    assert c.address == ctypes.addressof(c.struct) and bytes(c.struct) == bytes(plan.struct)
    assert (c.n_axes, c.head_dim) == (plan.n_axes, plan.head_dim) == (3, 128)
    want, address = bytes(plan.struct), c.address
    del a, plan
    gc.collect()
    assert ctypes.string_at(address, len(want)) == want
    if how is not copy.copy:
        assert how({"plan": c})["plan"].address != c.address
    assert zl._lib.load().zl_rope_fwd(c.ref, 64, 128, 64, 128, 64, 10, 0, 1, 1, _lib.ZL_BF16, 64, 128, 64, 128,
                                      None) == _lib.ZL_OK


def test_lists_and_sizes_past_32_bits_are_refused():
    for bad in ([0, 2**32 + 5], [0, -2**32], [0, 2**31]):
        with pytest.raises(ValueError, match="32 bits"):
            zl.host_int32(bad)
        with pytest.raises(ValueError, match="32 bits"):
            zl.fwd_workspace_bytes(bad, [0, 5], 4, 64)
    assert list(zl.host_int32([-2**31, 2**31 - 1])) == [-2**31, 2**31 - 1]
    with pytest.raises(ValueError, match="32 bits"):
        zl.RopePlan(64, axes=(2**32 + 64,))
    for args, name in ((([0, 1], 16, 2**32 + 8, 8, 64), "num_heads"), (([0, 1], 16, 8, 2**32 + 8, 64), "num_kv_heads"),
                       (([0, 1], 16, 8, 8, 2**32 + 64), "head_dim")):
        with pytest.raises(ValueError, match=name):
            zl.paged_attn_workspace_bytes(*args)
    meta = lambda *s, dtype=torch.int32: torch.empty(s, dtype=dtype, device="meta")   # shapes without memory
    cache, long = meta(1, 1, 16, 64, dtype=torch.bfloat16), meta(2**32 + 1)
    with pytest.raises(ValueError, match="length of src"):
        zl.pages_copy(cache, long, long)
    with pytest.raises(ValueError, match="length of slots"):
        zl.pages_free(meta(2, 4), meta(2), meta(8), long, 16)
    with pytest.raises(ValueError, match="number of pages"):
        zl.pages_extend(meta(2, 4), meta(2), long, meta(2), 16)
    with pytest.raises(ValueError, match="columns"):
        zl.pages_truncate(meta(2, 2**31), meta(2), meta(8), meta(2), 16)


def test_attn_bounds_whose_last_block_ends_past_32_bits(lib):
    arr, n = _lib.int32_array([0, 3])
    c = _cache(table_cols=2**27 - 1)                  # a row holds 2^31 - 16 tokens
    out = ctypes.c_size_t(0)
    for most in (2**31 - 256, 2**31 - 17):
        assert lib.zl_paged_attn_workspace_size(arr, n - 1, most, 4, 2, 64, ctypes.byref(out)) == _lib.ZL_EINVAL
        assert lib.zl_paged_attn(ctypes.byref(c), P64, 256, arr, n - 1, most, 4, 0.125, 1, 0, P64, P64, P64, 1 << 40,
                                 None) == _lib.ZL_EINVAL
    assert lib.zl_paged_attn_workspace_size(arr, n - 1, 2**31 - 257, 4, 2, 64, ctypes.byref(out)) == _lib.ZL_OK


@pytest.mark.parametrize("kw", [{"factor": 1e-320}, {"factor": 1e-320, "ramp": (1.0, 4.0, 1.0)}, {"magnitude": 1e-60},
                                {"magnitude": -1e-60}, {"magnitude": float("nan")}])
def test_plans_whose_numbers_overflow_or_vanish(kw):
    with pytest.raises(zl.ZlError) as e:
        zl.RopePlan(64, **kw)
    assert e.value.status == _lib.ZL_EINVAL


def test_every_entry_is_declared_to_ctypes(lib):
    """No call falls back on what ctypes makes of undeclared arguments."""
    for name in _lib.EXPORTS:
        fn = getattr(lib, name)
        assert fn.argtypes is not None, name
        assert fn.restype in (ctypes.c_int32, ctypes.c_int64, ctypes.c_char_p), name


def test_a_binding_of_another_pytorch_is_refused_and_rebuilt(monkeypatch):
    from mixed_length_dit_gb300 import build
    assert _lib.bind().torch_version == torch.__version__
    monkeypatch.setattr(_lib, "_bind", None)
    monkeypatch.setattr(torch, "__version__", "1.0")
    with pytest.raises(RuntimeError, match="built for .* this is 1.0: run"):
        _lib.bind()
    with pytest.raises(RuntimeError, match="built for"):
        zl.paged_append(_b(1, 1, 64), _b(1, 1, 64), _b(1, 1, 16, 64), _b(1, 1, 16, 64), _i(1, 1), _i(1), [0, 1])
    assert not build._bind_stale(0.0)
    monkeypatch.setattr(build, "_torch_version", lambda: "1.0")
    assert build._bind_stale(0.0)
