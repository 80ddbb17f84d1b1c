"""The operators around a paged key/value cache, as a user's program calls them.

Four kinds of cases:

  rope    rotary positions of packed queries and keys, forward and backward
  append  new tokens' keys (rotated) and values into the cache's pages, with the queries rotated beside them
  attn    attention of a chunk of new tokens (down to single ones) over the paged cache
  pages   what a generation loop does with whole pages: extending, forking and compacting sequences

A cache is a pool of pages [P, Hk, page, d] for keys and one for values, a table of page numbers per sequence, the
sequences' lengths and a count of references per page.  The lengths count the new tokens as well.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def _rope(name, direction, tokens, heads, kv_heads, dim, axes, interleaved, dtype="bf16", base=10000.0, factor=1.0,
          ramp=False, fused=False, start=0):
    return {"name": name, "op": "rope", "dir": direction, "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "axes": axes, "interleaved": interleaved, "dtype": dtype, "base": base, "factor": factor,
            "ramp": ramp, "fused": fused, "start": start}


def _append(name, seqs, new_lo, new_hi, past_lo, past_hi, heads, kv_heads, dim, page, interleaved=False):
    return {"name": name, "op": "append", "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo,
            "past_hi": past_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "interleaved": interleaved}


def _attn(name, seqs, new_lo, new_hi, past_lo, past_hi, heads, kv_heads, dim, page, causal=True, window=0):
    return {"name": name, "op": "attn", "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo,
            "past_hi": past_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "causal": causal,
            "window": window}


def _pages(name, kind, slots, len_lo, len_hi, kv_heads, dim, page, groups, count):
    return {"name": name, "op": "pages", "kind": kind, "slots": slots, "len_lo": len_lo, "len_hi": len_hi,
            "kv_heads": kv_heads, "dim": dim, "page": page, "groups": groups, "count": count}


def listed():
    return [
        # q and k of the image mix (16 x 256, 8 x 1,024 and 4 x 4,096 tokens), just before the forward
        _rope("rope_fwd_images", "fwd", 28672, 24, 24, 128, "128", True),
        # gradients of the large training step (190,288 tokens, 40 heads) with frame/row/column positions
        _rope("rope_bwd_video_step", "bwd", 190288, 40, 40, 128, "44+42+42", True),
        # a few sequences of a fused q/k/v projection, shared key heads, half of each head rotated, far positions
        _rope("rope_fwd_long_part", "fwd", 1531, 32, 8, 128, "64", False, base=500000.0, factor=8.0, ramp=True,
              fused=True, start=900001),
        # one token for each sequence of a serving batch
        _append("append_single", 64, 1, 1, 500, 4000, 40, 8, 128, 16),
        # a ragged batch of prompt chunks
        _append("append_chunks", 12, 500, 4001, 0, 9000, 24, 24, 128, 64, interleaved=True),
        # the smallest call: one sequence's next token
        _attn("attn_one_token", 1, 1, 1, 1000, 1000, 24, 8, 128, 16),
        # a serving batch's next tokens over long ragged caches
        _attn("attn_tokens_long", 48, 1, 1, 1500, 16384, 40, 8, 128, 16),
        # a few drafted tokens a sequence, every head with keys of its own, head dimension 64
        _attn("attn_draft_mha", 9, 2, 7, 700, 9001, 16, 16, 64, 32),
        # prompt chunks over what is cached, causal, shared key heads
        _attn("attn_prompt_chunks", 3, 1000, 2048, 2000, 8192, 40, 8, 128, 64),
        # three latent frames of 480p (1,560 tokens each) over the 21-frame video's cache, all keys seen
        _attn("attn_video_chunk", 1, 4680, 4680, 28080, 28080, 24, 24, 128, 128, causal=False),
        # every sequence forked once, as a search or a set of samples does
        _pages("pages_fork", "fork", 64, 200, 5000, 8, 128, 16, 8, 32),
        # a pool with holes packed to its front
        _pages("pages_compact", "compact", 96, 100, 6000, 8, 128, 16, 16, 0),
    ]


def draw(rng):
    """One more case; sizes over their whole ranges, by their logarithm."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def heads():
        kv = rng.choice((1, 2, 3, 4, 8, 10))
        return kv * rng.choice((1, 2, 3, 4, 5, 8)), kv

    op = rng.choice(("rope", "append", "attn", "attn", "pages"))
    if op == "rope":
        dim = rng.choice((64, 128))
        h, kv = heads()
        axes = rng.choice({64: ("64", "32", "22+20+22"), 128: ("128", "64", "44+42+42", "96")}[dim])
        one = "+" not in axes
        c = _rope("", rng.choice(("fwd", "bwd")), log(1, 100000), h, kv, dim, axes, rng.random() < 0.5,
                  dtype=rng.choice(("bf16", "bf16", "fp32")), base=rng.choice((10000.0, 500000.0)),
                  factor=rng.choice((1.0, 4.0)), ramp=one and rng.random() < 0.4, fused=rng.random() < 0.4,
                  start=rng.randrange(1000000) if one else 0)
    elif op == "append":
        h, kv = heads()
        hi = log(1, 4000)
        past = log(1, 9000)
        c = _append("", log(1, 24), max(1, hi // rng.randint(1, 4)), hi, past // rng.randint(1, 6), past, h, kv,
                    rng.choice((64, 128)), rng.choice((16, 32, 64, 128)), rng.random() < 0.5)
    elif op == "attn":
        h, kv = heads()
        if rng.random() < 0.6:      # single tokens and drafts
            hi = rng.choice((1, 1, 1, 2, 5, 9))
            seqs, past = log(1, 48), log(16, 16000)
        else:                       # chunks
            hi = log(16, 2000)
            seqs, past = log(1, 3), log(1, 8000)
        dim = rng.choice((64, 128))
        win = rng.choice((0, 0, 0, log(8, 4096)))
        c = _attn("", seqs, rng.choice((1, max(1, hi // rng.randint(1, 3)))), hi, past // rng.randint(1, 8), past, h, kv, dim,
                  rng.choice((16, 32, 64, 128)), causal=win > 0 or rng.random() < 0.8, window=win)
    else:
        kind = rng.choice(("fork", "compact", "extend"))
        hi = log(16, 5000)
        slots = log(4, 64)
        c = _pages("", kind, slots, hi // rng.randint(1, 8), hi, rng.choice((1, 2, 4, 8)), rng.choice((64, 128)),
                   rng.choice((16, 32, 64)), log(1, 8), rng.randint(1, max(1, slots // 2)))
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes that a case stands for
def _spread(n, lo, hi, step=40503):
    """n lengths over [lo, hi], the last of them hi: the same ones for every seed."""
    return [lo + (i * step % 65536) * (hi - lo) // 65536 for i in range(1, n)] + [hi]


def _lens(case):
    """New tokens and lengths (with the new tokens) of a case's sequences."""
    new = _spread(case["seqs"], case["new_lo"], case["new_hi"])
    past = _spread(case["seqs"], case["past_lo"], case["past_hi"], 24109)
    return new, [n + p for n, p in zip(new, past)]


def _pairs(case):
    """(query, key) pairs of the mask, and the keys that any query of each sequence sees."""
    pairs = keys = 0
    for n, length in zip(*_lens(case)):
        lo = [max(0, p - case["window"] + 1) if case["window"] else 0 for p in range(length - n, length)]
        hi = [p + 1 if case["causal"] else length for p in range(length - n, length)]
        pairs += sum(b - a for a, b in zip(lo, hi))
        keys += hi[-1] - lo[0]
    return pairs, keys


def _pool(case):
    """Lengths, pages per sequence, pages in the pool and live pages beyond the packed front, of a `pages` case."""
    lens = _spread(case["slots"], case["len_lo"], case["len_hi"])
    used = [-(-n // case["page"]) for n in lens]
    live = sum(used)
    extra = case["slots"] + 3 if case["kind"] != "extend" else sum(-(-c // case["page"]) + 1 for c in _counts(case))
    total = live + live // 2 + extra
    return lens, used, total, live - live * live // total


def _counts(case):
    return _spread(case["slots"], 0, max(1, case["len_hi"] // 3), 30011)


def work(case):
    if case["op"] == "rope":
        size = 2 if case["dtype"] == "bf16" else 4
        values = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * size * values + 4 * case["tokens"] * len(case["axes"].split("+")), "flops": 3 * values}
    if case["op"] == "append":
        tokens = sum(_lens(case)[0])
        values = tokens * (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
        return {"bytes": 4 * values, "flops": 3 * tokens * (case["heads"] + case["kv_heads"]) * case["dim"]}
    if case["op"] == "attn":
        pairs, keys = _pairs(case)
        tokens = sum(_lens(case)[0])
        return {"bytes": 4 * tokens * case["heads"] * case["dim"] + 4 * tokens * case["heads"]
                + 4 * keys * case["kv_heads"] * case["dim"],
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    lens, used, total, moved = _pool(case)
    page_bytes = 2 * case["groups"] * case["kv_heads"] * case["page"] * case["dim"]
    if case["kind"] == "compact":
        return {"bytes": 2 * moved * page_bytes + 8 * (total + sum(used)), "flops": 0}
    if case["kind"] == "fork":
        tails = sum(lens[i] % case["page"] != 0 for i in range(case["count"]))
        return {"bytes": 2 * tails * page_bytes + 8 * (total + sum(used[: case["count"]])), "flops": 0}
    return {"bytes": 8 * total + 4 * sum(-(-c // case["page"]) for c in _counts(case)) + 12 * case["slots"], "flops": 0}


# ------------------------------------------------------------------ inputs
def _ramp(case):
    return (1.0, 4.0, 8192) if case["ramp"] else None


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    state = {"case": case}

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device=DEV)

    if case["op"] == "rope":
        tokens, h, kv, dim = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        dtype = DTYPES[case["dtype"]]
        if case["fused"]:       # q and k are parts of one projection's rows
            rows = normal(tokens, h + 2 * kv, dim, dtype=dtype)
            state["q"], state["k"] = rows[:, :h], rows[:, h:h + kv]
        else:
            state["q"], state["k"] = normal(tokens, h, dim, dtype=dtype), normal(tokens, kv, dim, dtype=dtype)
        at = torch.arange(tokens, device=DEV)
        if "+" in case["axes"]:  # frame, row and column of 480p latents
            pos = torch.stack((at // 1560, at // 52 % 30, at % 52))
            pos[0] += rng.randrange(64)
        else:
            pos = at[None] + case["start"] + rng.randrange(64)
        state["pos"] = pos.to(torch.int32).contiguous()
        return state

    if case["op"] in ("append", "attn"):
        new, lens = _lens(case)
        h, kv, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
        used = [-(-n // page) for n in lens]
        pool = sum(used) + 5
        numbers = list(range(pool))
        rng.shuffle(numbers)     # a cache in use: a sequence's pages lie anywhere
        table, at = [], 0
        for n in used:
            table.append(numbers[at:at + n] + [-1] * (max(used) - n))
            at += n
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        state.update(new=new, lens=lens, cu=cu, max_len=max(lens), table=whole(table), kv_lens=whole(lens))
        state["q"] = normal(cu[-1], h, dim)
        state["k_pages"], state["v_pages"] = normal(pool, kv, page, dim), normal(pool, kv, page, dim)
        if case["op"] == "append":
            state["k"], state["v"] = normal(cu[-1], kv, dim), normal(cu[-1], kv, dim)
        return state

    lens, used, total, moved = _pool(case)
    kind, live = case["kind"], sum(used)
    front = list(range(live))
    back = list(range(live, total))
    rng.shuffle(front)
    rng.shuffle(back)
    numbers = front[:live - moved] + back[:moved]
    rng.shuffle(numbers)
    most = max(used) + 2 + max(-(-c // case["page"]) for c in _counts(case))
    refs, table, at = [0] * total, [], 0
    for n in used:
        table.append(numbers[at:at + n] + [-1] * (most - n))
        for p in numbers[at:at + n]:
            refs[p] += 1
        at += n
    if kind == "fork":           # as many free slots as are forked
        table += [[-1] * most for _ in range(case["count"])]
        children = list(range(case["slots"], case["slots"] + case["count"]))
        rng.shuffle(children)
        state["parents"], state["children"] = whole(list(range(case["count"]))), whole(children)
        lens = lens + [0] * case["count"]
    state.update(table=whole(table), lens=whole(lens), refs=whole(refs), counts=whole(_counts(case)))
    if kind != "extend":
        state["cache"] = normal(case["groups"], total, case["kv_heads"], case["page"], case["dim"])
    return state


# ------------------------------------------------------------------ the plain forms
def _frequencies(case):
    """Angle per position of each rotated pair, in 64 bits, and the axis whose position it takes."""
    freq, axis = [], []
    for a, d in enumerate(int(x) for x in case["axes"].split("+")):
        f = case["base"] ** (-torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / d)
        if case["ramp"]:
            low, high, length = _ramp(case)
            keep = ((f * length / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
            f = f * (keep + (1 - keep) / case["factor"])
        else:
            f = f / case["factor"]
        freq.append(f)
        axis.append(torch.full((d // 2,), a, device=DEV))
    return torch.cat(freq), torch.cat(axis)


def _rotate(x, pos, case, sign):
    """x [T, heads, dim] with its first pairs rotated by sign * (their positions' angles)."""
    freq, axis = _frequencies(case)
    half = freq.numel()
    angle = pos.double().T[:, axis] * freq
    cos, sin = angle.cos().float()[:, None], sign * angle.sin().float()[:, None]
    y = x.float()
    if case["interleaved"]:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, y[..., 2 * half:]), -1).to(x.dtype)


def _append_rope(case):
    return {"axes": str(case["dim"]), "base": 10000.0, "factor": 1.0, "ramp": False,
            "interleaved": case["interleaved"]}


def _places(state):
    """Of each new token: its sequence and its position."""
    n = torch.tensor(state["new"], device=DEV)
    seq = torch.repeat_interleave(torch.arange(len(state["new"]), device=DEV), n, output_size=state["cu"][-1])
    start = torch.tensor(state["cu"][:-1], device=DEV)
    at = torch.arange(state["cu"][-1], device=DEV) - start[seq]
    return seq, at, state["kv_lens"].long()[seq] - n[seq] + at


def _plain_append(state):
    case = state["case"]
    seq, _, pos = _places(state)
    rope = _append_rope(case)
    q, k = _rotate(state["q"], pos[None], rope, 1), _rotate(state["k"], pos[None], rope, 1)
    page = state["table"].long()[seq, pos // case["page"]]
    state["k_pages"][page, :, pos % case["page"]] = k
    state["v_pages"][page, :, pos % case["page"]] = state["v"]
    return q, state["k_pages"], state["v_pages"]


def _plain_attn(state):
    case = state["case"]
    h, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    seqs, most, longest = len(state["new"]), max(state["new"]), state["max_len"]
    seq, at, pos = _places(state)
    q = torch.zeros(seqs, most, h, dim, device=DEV)
    q[seq, at] = state["q"].float()
    q = q.view(seqs, most, kv, h // kv, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv, h // kv * most, dim)
    table = state["table"].long().clamp(min=0)

    def cached(pages):
        return pages[table].transpose(2, 3).flatten(1, 2)[:, :longest].transpose(1, 2).float()

    score = (q @ cached(state["k_pages"]).mT).mul_(dim ** -0.5)
    lens = state["kv_lens"].long()[:, None, None]
    p = lens - torch.tensor(state["new"], device=DEV)[:, None, None] + torch.arange(most, device=DEV)[None, :, None]
    key = torch.arange(longest, device=DEV)[None, None]
    seen = (key < lens) & (p < lens)
    if case["causal"]:
        seen = seen & (key <= p)
    if case["window"]:
        seen = seen & (key > p - case["window"])
    score = score.view(seqs, h, most, longest).masked_fill_(~seen[:, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0]
    used = key < lens
    o = score.view(seqs, kv, h // kv * most, longest) @ cached(state["v_pages"]).masked_fill(~used[..., None].view(seqs, 1, longest, 1), 0)
    o = o.view(seqs, h, most, dim) / total
    return o.transpose(1, 2)[seq, at].to(state["q"].dtype), lse.transpose(1, 2)[seq, at].T.contiguous()


def _plain_pages(state):
    case = state["case"]
    page = case["page"]
    table, lens, refs = state["table"].clone(), state["lens"].clone(), state["refs"].clone()
    column = torch.arange(table.shape[1], device=DEV)
    if case["kind"] == "extend":
        grown = lens + state["counts"]
        had, needs = (lens + page - 1) // page, (grown + page - 1) // page
        fresh = (column >= had[:, None]) & (column < needs[:, None])
        free = (refs == 0).nonzero()[:, 0][:int(fresh.sum())]
        table[fresh] = free.to(torch.int32)
        refs[free] = 1
        return table, grown, refs
    cache = state["cache"]
    if case["kind"] == "fork":
        parents, children = state["parents"].long(), state["children"].long()
        length = lens[parents]
        rows = table[parents]
        kept = column < (length // page)[:, None]
        tails = (length % page != 0).nonzero()[:, 0]
        at = (length // page)[tails].long()
        free = (refs == 0).nonzero()[:, 0][:tails.numel()]
        cache[:, free] = cache[:, rows[tails, at].long()]
        refs.index_add_(0, rows[kept].long(), torch.ones_like(rows[kept]))
        refs[free] = 1
        rows = torch.where(kept, rows, table[children])
        rows[tails, at] = free.to(torch.int32)
        table[children] = rows
        lens[children] = length
        return cache, table, lens, refs
    live = (refs > 0).sum()
    number = torch.arange(refs.numel(), device=DEV)
    source = ((refs > 0) & (number >= live)).nonzero()[:, 0]
    target = ((refs == 0) & (number < live)).nonzero()[:, 0]
    cache[:, target] = cache[:, source]
    moved = number.to(torch.int32)
    moved[source] = target.to(torch.int32)
    refs[target] = refs[source]
    refs[source] = 0
    in_row = column < ((lens + page - 1) // page)[:, None]
    table = torch.where(in_row, moved[table.long().clamp(min=0)], table)
    return cache, table, lens, refs


# ------------------------------------------------------------------ the framework's calls
def _own_rope(state):
    import mixed_length_dit_gb300 as zl
    case = state["case"]
    if "plan" not in state:
        state["plan"] = zl.RopePlan(case["dim"], axes=tuple(int(x) for x in case["axes"].split("+")), base=case["base"],
                                    interleaved=case["interleaved"], factor=case["factor"], ramp=_ramp(case))
    turn = zl.rope_fwd if case["dir"] == "fwd" else zl.rope_bwd
    return turn(state["q"], state["k"], state["pos"], state["plan"])


def _own_append(state):
    import mixed_length_dit_gb300 as zl
    case = state["case"]
    if "plan" not in state:
        state["plan"] = zl.RopePlan(case["dim"], interleaved=case["interleaved"])
        state["batch"] = zl.host_int32(state["cu"])
    q = zl.paged_append(state["k"], state["v"], state["k_pages"], state["v_pages"], state["table"], state["kv_lens"],
                        state["batch"], q=state["q"], rope=state["plan"])
    return q, state["k_pages"], state["v_pages"]


def _own_attn(state):
    import mixed_length_dit_gb300 as zl
    case = state["case"]
    if "batch" not in state:
        state["batch"] = zl.host_int32(state["cu"])
        state["workspace"] = zl.alloc_workspace(zl.paged_attn_workspace_bytes(
            state["batch"], state["max_len"], case["heads"], case["kv_heads"], case["dim"]), DEV)
    return zl.paged_attn(state["q"], state["k_pages"], state["v_pages"], state["table"], state["kv_lens"],
                         state["batch"], state["max_len"], causal=case["causal"], window=case["window"],
                         workspace=state["workspace"])


def _own_pages(state):
    import mixed_length_dit_gb300 as zl
    case = state["case"]
    table, lens, refs = state["table"].clone(), state["lens"].clone(), state["refs"].clone()
    if case["kind"] == "extend":
        zl.pages_extend(table, lens, refs, state["counts"], case["page"])
        return table, lens, refs
    if "workspace" not in state:
        state["workspace"] = zl.alloc_workspace(zl.pages_workspace_bytes(refs.numel()), DEV)
    if case["kind"] == "fork":
        zl.pages_fork(state["cache"], table, lens, refs, state["parents"], state["children"],
                      workspace=state["workspace"])
    else:
        zl.pages_compact(state["cache"], table, lens, refs, workspace=state["workspace"])
    return state["cache"], table, lens, refs


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "attn": _own_attn, "pages": _own_pages}[op](state)
    if op == "rope":
        sign = 1 if state["case"]["dir"] == "fwd" else -1
        return tuple(_rotate(state[x], state["pos"], state["case"], sign) for x in ("q", "k"))
    return {"append": _plain_append, "attn": _plain_attn, "pages": _plain_pages}[op](state)


# ------------------------------------------------------------------ the definitions, in 64 bits
def _turned(x, pos, axes, base, interleaved, sign, factor=1.0, ramp=None):
    """x times the block-diagonal rotation, pair by pair; pos [axes, T]."""
    y = x.double().clone()
    half, i = sum(axes) // 2, 0
    for a, d in enumerate(axes):
        for j in range(d // 2):
            f = math.exp(-2.0 * j / d * math.log(base))
            if ramp is None:
                f /= factor
            else:
                turns = f * ramp[2] / (2 * math.pi)
                w = min(1.0, max(0.0, (turns - ramp[0]) / (ramp[1] - ramp[0])))
                f = w * f + (1 - w) * f / factor
            first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            z = torch.polar(torch.ones_like(pos[a], dtype=torch.float64), sign * f * pos[a].double())[:, None]
            z = z * torch.complex(x[..., first].double(), x[..., second].double())
            y[..., first], y[..., second] = z.real, z.imag
            i += 1
    return y


def exact(case, seed):
    if case["op"] == "pages":    # whole numbers and copies: nothing is computed
        return None
    state = prepare(case, seed)
    if case["op"] == "rope":
        axes = [int(x) for x in case["axes"].split("+")]
        sign = 1 if case["dir"] == "fwd" else -1
        return tuple(_turned(state[x], state["pos"], axes, case["base"], case["interleaved"], sign, case["factor"],
                             _ramp(case)) for x in ("q", "k"))
    new, lens, cu, page = state["new"], state["lens"], state["cu"], case["page"]
    if case["op"] == "append":
        pos = torch.cat([torch.arange(b - n, b, device=DEV) for n, b in zip(new, lens)])[None]
        q, k = (_turned(state[x], pos, [case["dim"]], 10000.0, case["interleaved"], 1) for x in ("q", "k"))
        pages = state["k_pages"].double(), state["v_pages"].double()
        for s, (n, b) in enumerate(zip(new, lens)):
            numbers = state["table"][s].tolist()
            for x, rows in zip(pages, (k, state["v"].double())):
                done = b - n
                while done < b:
                    stop = min(b, (done // page + 1) * page)
                    row = cu[s] + done - (b - n)
                    x[numbers[done // page], :, done % page:done % page + stop - done] = \
                        rows[row:row + stop - done].transpose(0, 1)
                    done = stop
        return (q,) + pages
    if work(case)["flops"] > 6e12:
        return None
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(state["q"].shape[1::-1], dtype=torch.float64, device=DEV)
    for s, (n, b) in enumerate(zip(new, lens)):
        numbers = state["table"][s, :-(-b // page)].long()
        p = torch.arange(b - n, b, device=DEV)[:, None]
        j = torch.arange(b, device=DEV)[None]
        hidden = torch.zeros(n, b, dtype=torch.bool, device=DEV)
        if case["causal"]:
            hidden |= j > p
        if case["window"]:
            hidden |= j <= p - case["window"]
        for g in range(case["kv_heads"]):
            k, v = (state[x][numbers, g].double().flatten(0, 1)[:b] for x in ("k_pages", "v_pages"))
            for i in range(g * group, (g + 1) * group):
                x = state["q"][cu[s]:cu[s + 1], i].double() @ k.T / math.sqrt(case["dim"])
                x[hidden] = -math.inf
                lse[i, cu[s]:cu[s + 1]] = torch.logsumexp(x, 1)
                out[cu[s]:cu[s + 1], i] = torch.softmax(x, 1) @ v
    return out, lse
