"""The compiled short way of the binding against the long one: the same bits,
taken for regular calls, from several threads, and errors as PyTorch's own."""
import threading

import pytest
import torch

import mixed_length_dit_gb300 as zl
from mixed_length_dit_gb300 import _lib

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Long:
    """Stands in for the compiled binding and declines every call."""

    def __getattr__(self, name):
        return lambda *args: None


class Counting:
    """Passes calls on, and counts those that the short way took."""

    def __init__(self):
        self.real, self.taken = _lib.bind(), []

    def __getattr__(self, name):
        def call(*args):
            r = getattr(self.real, name)(*args)
            if r is not None:
                self.taken.append(name)
            return r
        return call


def setup(seed=3, hd=128, heads=8, kv=2, page=32, slots=3, pages=24):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)
    cache = torch.zeros((2, pages, kv, page, hd), dtype=BF16, device="cuda")
    return {"plan": zl.RopePlan(hd), "cu": zl.host_int32([0, 40, 41, 46]), "counts": i32([40, 1, 5, 0, 0]),
            "qkv": rand(46, heads + 2 * kv, hd), "pos": torch.arange(46, dtype=torch.int32, device="cuda"),
            "cache": cache, "table": torch.full((slots + 2, 4), -1, dtype=torch.int32, device="cuda"),
            "lens": i32([0] * (slots + 2)), "refs": i32([0] * pages), "heads": heads, "kv": kv, "page": page}


def run(s):
    """Every operation that has a short way, on one cache; all that they leave."""
    h, kv = s["heads"], s["kv"]
    q, k, v = s["qkv"][:, :h], s["qkv"][:, h:h + kv], s["qkv"][:, h + kv:]
    out = list(zl.rope_fwd(q, k, s["pos"], s["plan"])) + list(zl.rope_bwd(q, k, s["pos"], s["plan"]))
    out += [zl.rope_fwd(q, None, s["pos"], s["plan"])[0]]
    out += [zl.pages_extend(s["table"], s["lens"], s["refs"], s["counts"], s["page"])]
    kp, vp = s["cache"]
    table, lens = s["table"][:3], s["lens"][:3]
    assert zl.paged_append(k, v, kp, vp, table, lens, s["cu"]) is None
    qr = zl.paged_append(k, v, kp, vp, table, lens, s["cu"], q=q, rope=s["plan"])
    out += [qr, *zl.paged_attn(qr, kp, vp, table, lens, s["cu"], 128)]
    ws = zl.alloc_workspace(zl.paged_attn_workspace_bytes(s["cu"], 128, h, kv, 128), "cuda")
    o, lse = torch.empty_like(out[-2]), torch.empty_like(out[-1])
    got = zl.paged_attn(qr, kp, vp, table, lens, s["cu"], 128, causal=False, window=30, softmax_scale=0.05, out=o,
                        lse=lse, workspace=ws)
    assert got[0].data_ptr() == o.data_ptr() and got[1].data_ptr() == lse.data_ptr()
    out += [o, lse]
    ws = zl.alloc_workspace(zl.pages_workspace_bytes(s["refs"].shape[0]), "cuda")
    out += [zl.pages_fork(s["cache"], s["table"], s["lens"], s["refs"], i32([0, 2]), i32([3, 4]), workspace=ws)]
    zl.pages_free(s["table"], s["lens"], s["refs"], i32([0]), s["page"])
    out += [zl.pages_compact(s["cache"], s["table"], s["lens"], s["refs"], workspace=ws)]
    zl.sync_check()
    return out + [s["cache"], s["table"], s["lens"], s["refs"]]


def test_both_ways_give_the_same_bits(monkeypatch):
    counting = Counting()
    monkeypatch.setattr(_lib, "_bind", counting)
    short = run(setup())
    assert sorted(counting.taken) == sorted(["rope"] * 3 + ["extend"] + ["append"] * 2 + ["attn"] * 2 +
                                            ["fork", "compact"])
    monkeypatch.setattr(_lib, "_bind", Long())
    long = run(setup())
    assert len(short) == len(long)
    for a, b in zip(short, long):
        assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride() and torch.equal(a, b)


@pytest.mark.parametrize("change", ["dtype", "strides", "shape", "devices", "positions"])
def test_unusual_calls_take_the_long_way(monkeypatch, change):
    counting = Counting()
    monkeypatch.setattr(_lib, "_bind", counting)
    q, pos, plan = torch.ones(6, 4, 64, device="cuda", dtype=BF16), i32([0] * 6), zl.RopePlan(64)
    error = ValueError
    if change == "dtype":
        q, error = q.to(torch.float16), TypeError
    elif change == "strides":
        q = q.transpose(0, 1).contiguous().transpose(0, 1)
    elif change == "shape":
        q = q[:, :, :32]
    elif change == "devices":
        pos = pos.cpu()
    else:
        pos = i32([[0] * 6, [0] * 6])
    with pytest.raises(error):
        zl.rope_fwd(q, None, pos, plan)
    assert counting.taken == []


def test_regular_calls_from_threads():
    want = run(setup())
    results, errors = {}, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                s = setup()
                results[i] = run(s)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for r in results.values():
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_without_memory_the_error_is_pytorchs():
    q, pos, plan = torch.ones(4096, 64, 64, device="cuda", dtype=BF16), i32([0] * 4096), zl.RopePlan(64)
    q = q.clone()                              # 32 MiB, more than what is left below
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    used = torch.cuda.memory_reserved()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((used + (8 << 20)) / total)
    try:
        with pytest.raises(torch.cuda.OutOfMemoryError):
            hold = [zl.rope_fwd(q, None, pos, plan) for _ in range(4)]
            del hold
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    got = zl.rope_fwd(q, None, pos, plan)[0]
    zl.sync_check()
    assert torch.equal(got, q)                 # position 0 turns by nothing
