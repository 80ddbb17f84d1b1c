"""The 4-bit cache without a GPU: facts about the oracle, and the refusals of the
C ABI and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

import mixed_length_dit_gb300 as zl
from mixed_length_dit_gb300 import _lib
from oracle import q4_f64 as q4
from test_paged_host import CACHE_FAULTS, P64, _cache

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


# ------------------------------------------------------------------ the oracle
def test_steps_are_halves_without_a_sign():
    b = np.arange(256, dtype=np.uint16)
    half = (b << 7).astype(np.uint16).view(np.float16).astype(np.float64)
    assert np.array_equal(q4.STEPS[:248], half[:248]) and np.isnan(q4.STEPS[248:]).all()
    assert np.all(np.diff(q4.STEPS[:248]) > 0) and q4.STEPS[247] == 61440


def test_a_step_is_its_groups_seventh_to_four_bits():
    for top in (7.0, 1.0, 0.3, 100.0, 1e-3, 7 * 61440.0):
        s = q4.step_of(q4.step_byte(top))
        assert abs(s - top / 7) <= top / 7 / 16                # half of the last of four bits, at most 1/16
    assert q4.step_of(q4.step_byte(7 * 17.0)) == 18            # a half goes up: 17 has five bits
    assert q4.step_of(q4.step_byte(7 * 19.0)) == 20
    assert q4.step_byte(0.0) == 0 and q4.step_byte(1e30) == 247
    assert q4.step_byte(float("inf")) == 255 and q4.step_byte(7 * 2.0 ** -14) == 8
    assert q4.step_byte(7 * 2.0 ** -17) == 1 and q4.step_byte(7 * 2.0 ** -18) == 1 and q4.step_byte(6.9 * 2.0 ** -18) == 0


def test_values_are_within_half_a_step_and_exact_in_bf16():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 128)) * np.exp2(rng.integers(-12, 12, (50, 1)))
    x = torch.tensor(x).to(BF16).double().numpy()
    codes, byte = q4.quantise(x)
    v = q4.values(codes, byte)
    assert np.all(np.abs(v - x) <= np.repeat(q4.STEPS[byte], 32, -1) / 2)
    assert np.array_equal(torch.tensor(v).to(BF16).double().numpy(), v)
    again = q4.quantise(v)
    assert np.all(np.abs(q4.values(*again) - v) <= np.repeat(q4.STEPS[again[1]], 32, -1) / 2)


def test_halves_go_up():
    x = np.zeros((1, 32))
    x[0, :6] = [7.0, 0.5, 1.5, -0.5, -1.5, 2.5]                # step 1
    codes, byte = q4.quantise(x)
    assert codes[0, :6].tolist() == [7, 1, 2, 0, -1, 3] and q4.STEPS[byte[0, 0]] == 1.0


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("keys", [True, False])
def test_every_column_has_a_place_of_its_own(hd, keys):
    at = {q4.place(j, hd, keys) for j in range(hd)}
    assert len(at) == hd and {b for b, _ in at} == set(range(hd // 2))
    rng = np.random.default_rng(1)
    codes, byte = rng.integers(-8, 8, (3, 16, hd)), rng.integers(0, 256, (3, 16, hd // 32))
    blocks = q4.pack(codes, byte, keys)
    assert blocks.shape == (3, 16 * zl.q4_row_bytes(hd)) and blocks.dtype == np.uint8
    c2, b2 = q4.unpack(blocks, 16, hd, keys)
    assert np.array_equal(codes, c2) and np.array_equal(byte, b2)


def test_infinities_and_nan_take_their_group_along():
    x = np.ones((3, 64))
    x[0, 3], x[1, 40], x[2, 0] = np.nan, np.inf, -np.inf
    v = q4.values(*q4.quantise(x))
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] > 0).all()
    assert np.isnan(v[1, 32:]).all() and np.isnan(v[2, :32]).all() and (v[1, :32] > 0).all()


# ------------------------------------------------------------------ the C ABI
def _append(lib, c, cu, k=P64, ks=128, v=P64, vs=128, plan=None, pos=None, ps=0, q=None, qs=0, nq=0, qo=None, qos=0,
            status=None):
    arr, n = _lib.int32_array(cu)
    return lib.zl_paged_append_q4(ctypes.byref(c) if c else None, k, ks, v, vs, arr, n - 1, plan, pos, ps, q, qs, nq, qo,
                                  qos, status, None)


def _read(lib, c, cu, k=P64, ks=128, v=P64, vs=128):
    arr, n = _lib.int32_array(cu)
    return lib.zl_paged_read_q4(ctypes.byref(c) if c else None, arr, n - 1, k, ks, v, vs, None)


def _attn(lib, c, cu, q=P64, qs=None, most=100, nh=4, scale=0.125, causal=1, window=0, o=P64, lse=P64, ws=P64,
          ws_bytes=1 << 40):
    arr, n = _lib.int32_array(cu)
    return lib.zl_paged_attn_q4(ctypes.byref(c) if c else None, q, nh * 64 if qs is None else qs, arr, n - 1, most, nh,
                                scale, causal, window, o, lse, ws, ws_bytes, None)


def _bytes(lib, cu, most, nh, nk, hd, window=0):
    arr, n = _lib.int32_array(cu)
    out = ctypes.c_size_t(7)
    return lib.zl_paged_attn_q4_workspace_size(arr, n - 1, most, nh, nk, hd, window, ctypes.byref(out)), out.value


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_bad_caches(lib, fault, status):
    c = _cache(**fault)
    nk = fault.get("num_kv_heads", 2) or 1
    assert _append(lib, c, [0, 3]) == status
    assert _read(lib, c, [0, 3]) == status
    assert _attn(lib, c, [0, 3], nh=4 * nk) == status


def test_append_refusals(lib):
    c, plan = _cache(), zl.RopePlan(64)
    assert _append(lib, None, [0, 1]) == _lib.ZL_EINVAL
    assert _append(lib, c, [0, 0]) == _lib.ZL_OK               # nothing to do
    assert _append(lib, c, [0, 3, 1]) == _lib.ZL_EINVAL
    assert _append(lib, c, [1, 3]) == _lib.ZL_EINVAL
    assert _append(lib, c, [0, 1], k=None) == _lib.ZL_EINVAL
    assert _append(lib, c, [0, 1], ks=64) == _lib.ZL_EINVAL
    assert _append(lib, c, [0, 1], vs=129) == _lib.ZL_EALIGN
    assert _append(lib, c, [0, 1], v=ctypes.c_void_p(72)) == _lib.ZL_EALIGN
    assert _append(lib, c, [0, 1], nq=2) == _lib.ZL_EINVAL     # heads without queries
    assert _append(lib, c, [0, 1], q=P64, qs=128, nq=2, qo=None) == _lib.ZL_EINVAL
    assert _append(lib, c, [0, 1], pos=P64, ps=1) == _lib.ZL_EINVAL            # positions without a plan
    assert _append(lib, c, [0, 1], plan=ctypes.byref(zl.RopePlan(128).struct)) == _lib.ZL_EINVAL
    assert _append(lib, c, [0, 1], plan=ctypes.byref(zl.RopePlan(64, axes=(32, 32)).struct)) == _lib.ZL_EINVAL
    assert _append(lib, c, [0, 1], plan=plan.ref, status=ctypes.c_void_p(66)) == _lib.ZL_EALIGN


def test_read_refusals(lib):
    c = _cache()
    assert _read(lib, None, [0, 1]) == _lib.ZL_EINVAL
    assert _read(lib, c, [0, 0]) == _lib.ZL_OK
    assert _read(lib, c, [0, 2, 1]) == _lib.ZL_EINVAL
    assert _read(lib, c, [0, 1], k=None) == _lib.ZL_EINVAL
    assert _read(lib, c, [0, 1], ks=127) == _lib.ZL_EINVAL
    assert _read(lib, c, [0, 1], vs=132) == _lib.ZL_EALIGN


def test_attn_refusals(lib):
    c = _cache()
    assert _attn(lib, None, [0, 1]) == _lib.ZL_EINVAL
    assert _attn(lib, c, [0, 0]) == _lib.ZL_OK
    assert _attn(lib, c, [0, 1], nh=3) == _lib.ZL_EINVAL
    assert _attn(lib, c, [0, 1], nh=512) == _lib.ZL_EUNSUPPORTED               # 256 heads of a key head
    assert _attn(lib, c, [0, 1], most=129) == _lib.ZL_EINVAL                   # more than the table holds
    assert _attn(lib, c, [0, 1], most=-1) == _lib.ZL_EINVAL
    assert _attn(lib, c, [0, 1], scale=0.0) == _lib.ZL_EINVAL
    assert _attn(lib, c, [0, 1], scale=float("nan")) == _lib.ZL_EINVAL
    assert _attn(lib, c, [0, 1], causal=2) == _lib.ZL_EINVAL
    assert _attn(lib, c, [0, 1], window=-1) == _lib.ZL_EINVAL
    assert _attn(lib, c, [0, 1], o=None) == _lib.ZL_EINVAL
    assert _attn(lib, c, [0, 1], lse=ctypes.c_void_p(66)) == _lib.ZL_EALIGN
    assert _attn(lib, c, [0, 1], qs=255) == _lib.ZL_EINVAL
    for cu in ([0, 1], [0, 128]):
        _, need = _bytes(lib, cu, 100, 4, 2, 64)
        assert need > 0
        assert _attn(lib, c, cu, ws=None) == _lib.ZL_EWORKSPACE
        assert _attn(lib, c, cu, ws_bytes=need - 1) == _lib.ZL_EWORKSPACE
        assert _attn(lib, c, cu, ws=ctypes.c_void_p(72)) == _lib.ZL_EALIGN


def test_workspace_sizes(lib):
    assert _bytes(lib, [0, 1], 100, 4, 3, 64)[0] == _lib.ZL_EINVAL
    assert _bytes(lib, [0, 1], 100, 4, 2, 80)[0] == _lib.ZL_EUNSUPPORTED
    assert _bytes(lib, [0, 1], 100, 4, 2, 64, -1)[0] == _lib.ZL_EINVAL
    assert _bytes(lib, [0, 0], 100, 4, 2, 64) == (_lib.ZL_OK, 0)
    # a chunk's keys and values in bf16, by the bound or the window, whichever is less
    whole, windowed, longer = (_bytes(lib, [0, 2000], n, 8, 8, 128, w)[1] for n, w in ((32768, 0), (32768, 1024), (65536, 0)))
    assert 32768 * 8 * 128 * 4 <= whole < 32768 * 8 * 128 * 4 + (64 << 20) and windowed < whole < longer
    assert _bytes(lib, [0, 2000], 32768, 8, 8, 128, 1 << 30)[1] == whole
    # many long sequences: 1 GiB of them at a time
    many = _bytes(lib, [2000 * i for i in range(31)], 32768, 8, 8, 128)[1]
    assert (1 << 29) < many < (1 << 30) + (64 << 20)
    assert _bytes(lib, [0, 2000], 2 ** 31 - 257, 8, 8, 128)[0] == _lib.ZL_EUNSUPPORTED


# ------------------------------------------------------------------ the binding
def _tensors(hd=128, page=16, kv=2, pages=9, seqs=2, cols=4):
    pools = [torch.zeros(pages, kv, page, zl.q4_row_bytes(hd), dtype=torch.uint8) for _ in range(2)]
    return [*pools, torch.zeros(seqs, cols, dtype=torch.int32), torch.ones(seqs, dtype=torch.int32)]


def _rows(t, kv=2, hd=128):
    return torch.zeros(t, kv, hd, dtype=BF16)


def test_row_bytes():
    assert zl.q4_row_bytes(128) == 68 and zl.q4_row_bytes(64) == 34
    with pytest.raises(ValueError):
        zl.q4_row_bytes(80)


def test_binding_refuses_other_pools():
    k, v, table, lens = _tensors()
    kv = _rows(2), _rows(2)
    q = torch.zeros(2, 4, 128, dtype=BF16)
    calls = (lambda c: zl.paged_append_q4(*kv, *c, [0, 1, 2]), lambda c: zl.paged_read_q4(*c, [0, 1, 2]),
             lambda c: zl.paged_attn_q4(q, *c, [0, 1, 2], 10))
    for call in calls:
        with pytest.raises(TypeError, match="uint8"):
            call((k.to(BF16), v.to(BF16), table, lens))
        with pytest.raises(ValueError, match="68"):
            call((k[..., :64].contiguous(), v[..., :64].contiguous(), table, lens))
        with pytest.raises(ValueError, match="contiguous"):
            call((k[..., ::1].transpose(1, 2), v, table, lens))
        with pytest.raises(ValueError, match="v_pages"):
            call((k, v[:-1], table, lens))
        with pytest.raises(ValueError, match="rows"):
            call((k, v, table[:1], lens))
        with pytest.raises(ValueError, match="kv_lens"):
            call((k, v, table, lens.long()))
        with pytest.raises(ValueError, match="CUDA"):
            call((k, v, table, lens))
    with pytest.raises(TypeError, match="bf16"):
        zl.paged_append(*kv, k, v, table, lens, [0, 1, 2])


def test_binding_refuses_other_rows():
    c = _tensors()
    k, v = _rows(3), _rows(3)
    with pytest.raises(ValueError, match="k must be"):
        zl.paged_append_q4(_rows(2), v, *c, [0, 1, 3])
    with pytest.raises(ValueError, match="v must be"):
        zl.paged_append_q4(k, v.float(), *c, [0, 1, 3])
    with pytest.raises(ValueError, match="contiguous"):
        zl.paged_append_q4(torch.zeros(3, 128, 2, dtype=BF16).transpose(1, 2), v, *c, [0, 1, 3])
    with pytest.raises(ValueError, match="without q"):
        zl.paged_append_q4(k, v, *c, [0, 1, 3], q_out=k)
    with pytest.raises(ValueError, match="rope"):
        zl.paged_append_q4(k, v, *c, [0, 1, 3], positions=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="status"):
        zl.paged_append_q4(k, v, *c, [0, 1, 3], status=torch.zeros(2, dtype=torch.int32))
    q = torch.zeros(3, 4, 128, dtype=BF16)
    with pytest.raises(ValueError, match="ends at"):
        zl.paged_attn_q4(q, *c, [0, 1, 2], 10)
    with pytest.raises(ValueError, match="32 bits"):
        zl.paged_attn_q4(q, *c, [0, 1, 3], 1 << 33)
    with pytest.raises(ValueError, match="32 bits"):
        zl.paged_attn_q4(q, *c, [0, 1, 3], 10, window=1 << 32)
    with pytest.raises(ValueError, match="at least one"):
        zl.paged_read_q4(*c, [])
