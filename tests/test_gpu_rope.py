"""Rotary positions on the GPU against the float64 definition.

Tolerance of an element y of pair (a, b): one rounding to the output type,
eps/2 * |y|, plus what the float32 cosine and sine carry: their argument is
rounded to 2^-25 half turns (pi * 2^-25 of an angle), sincospi is off by at
most 2 units of 2^-24, and two products and a sum round at 2^-24 each, all
times |a| + |b|: together below 2^-21 (|a| + |b|).
"""
import numpy as np
import pytest
import torch

import mixed_length_dit_gb300 as zl
from oracle import paged_f64 as ref
from _helpers import f64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _x(seed, *shape, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _check(got, x, pos, axes, sign, il, magnitude=1.0, **kw):
    want = ref.rope(f64(x), pos.cpu().numpy().reshape(len(axes), -1), axes, interleaved=il, magnitude=magnitude,
                    sign=sign, **kw)
    tol = torch.finfo(x.dtype).eps / 2 * np.abs(want) + 2.0 ** -21 * ref.rope_reach(f64(x), axes, il, magnitude)
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), float((err - tol).max())


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,nq,nk,hd,axes", [
    (1, 1, 1, 64, (64,)), (3, 5, 1, 128, (128,)), (64, 40, 8, 128, (64,)), (257, 24, 24, 128, (44, 42, 42)),
    (130, 7, 7, 64, (22, 20, 22)), (33, 4, 2, 128, (6,)), (10, 3, 3, 64, (2, 4, 6, 8)), (5000, 2, 1, 128, (96, 32)),
])
def test_forward_and_backward(tokens, nq, nk, hd, axes, dtype, il):
    q, k = _x(1, tokens, nq, hd, dtype=dtype), _x(2, tokens, nk, hd, dtype=dtype)
    rng = np.random.default_rng(3)
    pos = torch.tensor(rng.integers(0, 5000, (len(axes), tokens)), dtype=torch.int32, device="cuda")
    plan = zl.RopePlan(hd, axes=axes, interleaved=il, magnitude=1.25)
    for fn, sign in ((zl.rope_fwd, 1), (zl.rope_bwd, -1)):
        qo, ko = fn(q, k, pos, plan)
        zl.sync_check()
        _check(qo, q, pos, axes, sign, il, 1.25)
        _check(ko, k, pos, axes, sign, il, 1.25)


@pytest.mark.parametrize("pos", [[0, -1, 2 ** 31 - 1, -2 ** 31, 16777217, 999999, -123457]])
def test_far_and_negative_positions(pos):
    """Angles are exact at any int32 position."""
    x = _x(5, len(pos), 3, 128, dtype=F32)
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    got, none = zl.rope_fwd(x, None, p, zl.RopePlan(128))
    assert none is None
    # the float64 definition itself is off by 2^31 * 2^-53 of an angle at the ends: far below 2^-21
    _check(got, x, p, (128,), 1, False)


@pytest.mark.parametrize("kw", [dict(base=500000.0, factor=8.0), dict(factor=4.0, ramp=(1.0, 4.0, 8192)),
                                dict(factor=2.5, ramp=(0.0, 32.0, 4096), base=1000.0)])
def test_scaled_frequencies(kw):
    x = _x(6, 50, 2, 128, dtype=F32)
    p = torch.arange(50, dtype=torch.int32, device="cuda") * 2003
    got, _ = zl.rope_fwd(x, None, p, zl.RopePlan(128, axes=(96,), **kw))
    _check(got, x, p, (96,), 1, False, **kw)


@pytest.mark.parametrize("axes", [(128,), (64,), (6, 4)])
def test_parts_of_one_projection_in_place(axes):
    """q and k inside rows [q | k | v], turned where they are: v, and the
    columns past the rotated ones, keep their bits."""
    rows = _x(7, 37, 10, 128)
    before = rows.clone()
    p = torch.arange(37, dtype=torch.int32, device="cuda")
    plan = zl.RopePlan(128, axes=axes)
    pos = p if len(axes) == 1 else torch.stack([p] * len(axes))
    q, k = rows[:, :6], rows[:, 6:8]
    zl.rope_fwd(q, k, pos, plan, q_out=q, k_out=k)
    _check(q, before[:, :6], pos, axes, 1, False)
    _check(k, before[:, 6:8], pos, axes, 1, False)
    assert torch.equal(rows[:, 8:], before[:, 8:]) and torch.equal(rows[:, :, sum(axes):], before[:, :, sum(axes):])
    # the same as out of place, bit by bit
    qo, ko = zl.rope_fwd(before[:, :6], before[:, 6:8], pos, plan)
    assert torch.equal(qo, q) and torch.equal(ko, k)


def test_backward_is_the_transpose():
    """<g, R x> = <R^T g, x> over every column, in float32."""
    x, g = _x(8, 40, 2, 64, dtype=F32), _x(9, 40, 2, 64, dtype=F32)
    p = torch.arange(40, dtype=torch.int32, device="cuda") * 77
    plan = zl.RopePlan(64, axes=(48,), interleaved=True, magnitude=0.75)
    y, _ = zl.rope_fwd(x, None, p, plan)
    d, _ = zl.rope_bwd(g, None, p, plan)
    a, b = (g.double() * y.double()), (d.double() * x.double())
    # each side is a sum of products whose float32 factors are off by 2^-21 (|a|+|b|) + 2^-24 |y|
    bound = 2.0 ** -20 * float((g.abs().double() * 2 * x.abs().double().amax(-1, keepdim=True)).sum())
    assert abs(float(a.sum() - b.sum())) <= bound


def test_empty_and_outputs():
    plan = zl.RopePlan(64)
    q = torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    qo, ko = zl.rope_fwd(q, None, torch.empty(0, dtype=torch.int32, device="cuda"), plan)
    assert qo.shape == q.shape and ko is None
    q = _x(1, 6, 2, 64)
    out = torch.full((6, 5, 64), 7.0, dtype=BF16, device="cuda")
    p = torch.arange(6, dtype=torch.int32, device="cuda")
    r, _ = zl.rope_fwd(q, None, p, plan, q_out=out[:, 1:3])          # into a part of wider rows
    _check(r, q, p, (64,), 1, False)
    assert torch.all(out[:, 0] == 7) and torch.all(out[:, 3:] == 7)


def test_other_stream_and_graph():
    plan = zl.RopePlan(128)
    q, k = _x(1, 300, 8, 128), _x(2, 300, 2, 128)
    p = torch.arange(300, dtype=torch.int32, device="cuda")
    want = zl.rope_fwd(q, k, p, plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = zl.rope_fwd(q, k, p, plan, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    outs = [torch.zeros_like(q), torch.zeros_like(k)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        zl.rope_fwd(q, k, p, plan, q_out=outs[0], k_out=outs[1])
    p += 5
    g.replay()
    want = zl.rope_fwd(q, k, p, plan)
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_before_the_attention():
    """As a training step uses it: turn, attend, and bring the gradients back
    through the turn; against the float64 oracle of the whole."""
    import oracle
    cu = [0, 70, 200, 201]
    plan = zl.RopePlan(64, axes=(24, 20, 20), interleaved=True)
    q, k, v, do = (_x(i, 201, 2, 64) for i in range(4))
    pos = torch.stack([torch.arange(201, device="cuda") // d % m for d, m in ((50, 9), (10, 5), (1, 10))]).int()
    qr, kr = zl.rope_fwd(q, k, pos, plan)
    o, lse = zl.varlen_attn_fwd(qr, kr, v, cu)
    dq, dk, dv = zl.varlen_attn_bwd(qr, kr, v, o, lse, do, cu)
    dq, dk = zl.rope_bwd(dq, dk, pos, plan)
    zl.sync_check()
    turn = lambda x, sign: ref.rope(x, pos.cpu().numpy(), (24, 20, 20), interleaved=True, sign=sign)
    q64, k64 = turn(f64(q), 1), turn(f64(k), 1)
    want_o, _ = oracle.varlen_attn_fwd(q64, k64, f64(v), cu, cu)
    assert np.abs(f64(o) - want_o).max() <= 2e-2
    gq, gk, gv = oracle.varlen_attn_bwd(q64, k64, f64(v), f64(do), cu, cu)
    for got, want in ((dq, turn(gq, -1)), (dk, turn(gk, -1)), (dv, gv)):
        assert np.linalg.norm(f64(got) - want) <= 2e-2 * np.linalg.norm(want)
