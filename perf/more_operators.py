"""The operators of a paged key/value cache held in 4 bits, as a user's program calls them.

Three kinds of cases:

  append  new tokens' keys and values quantised into the cache's pages, and what the pages then hold read back
  read    whole cached sequences read back as packed bf16 rows
  attn    attention of a chunk of new tokens (down to single ones) over the cache

A cache is a pool of pages for keys and one for values, uint8 [P, Hk, page, 17 d / 32], a table of page numbers per
sequence and the sequences' lengths, which count the new tokens as well.  Every 32 columns of a token's head share a
step s, and a value x is held as the whole number c in [-8, 7] nearest to x / s (halves up), so that it reads c * s:

  s    max|x| / 7, rounded to four significant bits (halves up): a byte 8 e + m that stands for
       (8 + m) / 8 * 2^(e - 15), or for m / 8 * 2^-14 where e is 0; at most 61,440
  c    kept as c + 8 in four bits, eight to a 32-bit word, the first lowest

The bytes of a page's head are its tokens' codes, d / 2 bytes each, and behind them its tokens' steps, d / 32 bytes
each.  Of a token's codes the 32-bit words of keys (the 16-bit words of values) stand in the order that four (eight)
threads read them in: word q of piece c where the columns' order has word c of group q.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def _append(name, seqs, new_lo, new_hi, past_lo, past_hi, kv_heads, dim, page):
    return {"name": name, "op": "append", "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo,
            "past_hi": past_hi, "kv_heads": kv_heads, "dim": dim, "page": page}


def _read(name, seqs, len_lo, len_hi, kv_heads, dim, page):
    return {"name": name, "op": "read", "seqs": seqs, "new_lo": len_lo, "new_hi": len_hi, "past_lo": 0, "past_hi": 0,
            "kv_heads": kv_heads, "dim": dim, "page": page}


def _attn(name, seqs, new_lo, new_hi, past_lo, past_hi, heads, kv_heads, dim, page, causal=True, window=0):
    return {"name": name, "op": "attn", "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo,
            "past_hi": past_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "causal": causal,
            "window": window}


def listed():
    return [
        # one token for each sequence of a serving batch
        _append("append_single", 64, 1, 1, 500, 4000, 8, 128, 16),
        # a ragged batch of prompt chunks, every head with keys of its own
        _append("append_chunks", 12, 500, 4001, 0, 9000, 24, 128, 64),
        # drafted tokens, head dimension 64
        _append("append_drafts", 9, 2, 7, 700, 9001, 16, 64, 32),
        # one short sequence taken out of the cache
        _read("read_short", 1, 1531, 1531, 8, 128, 16),
        # a serving batch's long ragged sequences
        _read("read_long", 24, 1500, 16384, 8, 128, 64),
        # the smallest call: one sequence's next token
        _attn("attn_one_token", 1, 1, 1, 1000, 1000, 24, 8, 128, 16),
        # a serving batch's next tokens over long ragged caches
        _attn("attn_tokens_long", 48, 1, 1, 1500, 16384, 40, 8, 128, 16),
        # one sequence as long as the longest video, whose next token all SMs share
        _attn("attn_one_long", 1, 1, 1, 131071, 131071, 40, 8, 128, 64),
        # a few drafted tokens a sequence, every head with keys of its own, head dimension 64
        _attn("attn_draft_mha", 9, 2, 7, 700, 9001, 16, 16, 64, 32),
        # drafts of shared key heads, each query over the last 4,096 keys
        _attn("attn_draft_window", 16, 3, 8, 2000, 12000, 32, 8, 128, 32, window=4096),
        # prompt chunks over what is cached, causal, shared key heads
        _attn("attn_prompt_chunks", 3, 1000, 2048, 2000, 8192, 40, 8, 128, 64),
        # three latent frames of 480p (1,560 tokens each) over the 21-frame video's cache, all keys seen
        _attn("attn_video_chunk", 1, 4680, 4680, 28080, 28080, 24, 24, 128, 128, causal=False),
    ]


def draw(rng):
    """One more case; sizes over their whole ranges, by their logarithm."""
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("append", "read", "attn", "attn", "attn"))
    kv, dim, page = rng.choice((1, 2, 3, 4, 8, 10)), rng.choice((64, 128)), rng.choice((16, 32, 64, 128, 256))
    if op == "append":
        hi, past = log(1, 4000), log(1, 9000)
        c = _append("", log(1, 24), max(1, hi // rng.randint(1, 4)), hi, past // rng.randint(1, 6), past, kv, dim, page)
    elif op == "read":
        hi = log(1, 16000)
        c = _read("", log(1, 24), max(1, hi // rng.randint(1, 8)), hi, kv, dim, page)
    else:
        kind = rng.random()
        if kind < 0.5:              # single tokens and drafts
            hi = rng.choice((1, 1, 1, 2, 5, 9))
            seqs, past = log(1, 48), log(16, 16000)
        elif kind < 0.75:           # a few rows to some hundred
            hi, seqs, past = log(8, 200), log(1, 8), log(16, 9000)
        else:                       # chunks
            hi, seqs, past = log(200, 2000), log(1, 2), log(1, 8000)
        win = rng.choice((0, 0, 0, log(8, 4096)))
        c = _attn("", seqs, rng.choice((1, max(1, hi // rng.randint(1, 3)))), hi, past // rng.randint(1, 8), past,
                  kv * rng.choice((1, 2, 3, 4, 5, 8)), kv, dim, page, causal=win > 0 or rng.random() < 0.8, window=win)
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


def work(case):
    tokens = sum(_lens(case)[0])
    row = case["kv_heads"] * case["dim"]             # of keys, or of values
    held = 2 * row * 17 // 32
    if case["op"] == "append":                       # rows in, what they are held as, and their values out
        return {"bytes": tokens * (4 * row + held + 4 * row), "flops": 6 * tokens * row}
    if case["op"] == "read":
        return {"bytes": tokens * (held + 4 * row), "flops": 2 * tokens * row}
    pairs, keys = _pairs(case)
    return {"bytes": 4 * tokens * case["heads"] * case["dim"] + 4 * tokens * case["heads"] + keys * held,
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ------------------------------------------------------------------ a pool's bytes
def _codes(pool, dim):
    """The codes [P, Hk, page, d / 2] and the steps [P, Hk, page, d / 32] of a pool, as views of it."""
    pages, heads, page, row = pool.shape
    flat = pool.view(pages, heads, page * row)
    cut = page * dim // 2
    return flat[..., :cut].unflatten(-1, (page, dim // 2)), flat[..., cut:].unflatten(-1, (page, dim // 32))


def _quantised(x):
    """Codes in [0, 15] of x [..., d] and the bytes of its steps [..., d / 32]."""
    y = x.float().unflatten(-1, (-1, 32))
    top = y.abs().amax(-1)
    want = top / 7
    # four significant bits: the float32's exponent and three bits of its mantissa, rounded at the next one
    normal = (((want.view(torch.int32) + (1 << 19)) >> 20) - (112 << 3)).clamp(max=0xf7)
    small = (want * 2.0 ** 17 + 0.5).floor().to(torch.int32)
    byte = torch.where(want >= 2.0 ** -14, normal, small)
    byte = torch.where(torch.isfinite(y).all(-1), byte, 0xff)
    step = _step(byte)[..., None]
    code = torch.where((step > 0) & torch.isfinite(step), (y / step + 0.5).floor().clamp(-8, 7), 0.0) + 8
    return code.to(torch.uint8).flatten(-2), byte.to(torch.uint8)


def _step(byte):
    """The step that a byte stands for, in float32."""
    b = byte.to(torch.int32)
    normal = ((b << 20) + (112 << 23)).view(torch.float32)
    return torch.where(b < 248, torch.where(b >= 8, normal, b.float() * 2.0 ** -17), math.nan)


def _packed(code, keys):
    """Codes [..., d] as the bytes of a token [..., d / 2]."""
    b = code[..., 0::2] | code[..., 1::2] << 4
    pieces, size = (4, 4) if keys else (8, 2)
    return b.unflatten(-1, (-1, pieces, size)).transpose(-2, -3).flatten(-3)


def _unpacked(held, step, keys):
    """Values [..., d] in float32 of a token's bytes [..., d / 2] and steps [..., d / 32]."""
    pieces, size = (4, 4) if keys else (8, 2)
    b = held.unflatten(-1, (pieces, -1, size)).transpose(-2, -3).flatten(-3)
    code = torch.stack((b & 15, b >> 4), -1).flatten(-2).unflatten(-1, (-1, 32))
    return ((code.float() - 8) * _step(step)[..., None]).flatten(-2)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)

    def whole(values):
        return torch.tensor(values, dtype=torch.int32, device=DEV)

    new, lens = _lens(case)
    kv, dim, page = case["kv_heads"], case["dim"], case["page"]
    used = [-(-n // page) for n in lens]
    pool = sum(used) + 5
    numbers = list(range(pool))
    rng.shuffle(numbers)             # a cache in use: a sequence's pages lie anywhere
    table, at = [], 0
    for n in used:
        table.append(numbers[at:at + n] + [-1] * (max(used) - n))
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    state = {"case": case, "new": new, "lens": lens, "cu": cu, "max_len": max(lens), "table": whole(table),
             "kv_lens": whole(lens)}
    for name in ("k", "v"):
        pages = torch.empty(pool, kv, page, dim * 17 // 32, dtype=torch.uint8, device=DEV)
        held, steps = _codes(pages, dim)
        for p in range(0, pool, 4096):
            code, byte = _quantised(normal(min(4096, pool - p), kv, page, dim))
            held[p:p + 4096] = _packed(code, name == "k")
            steps[p:p + 4096] = byte
        state[name + "_pages"] = pages
    if case["op"] == "append":
        state["k"], state["v"] = normal(cu[-1], kv, dim), normal(cu[-1], kv, dim)
    if case["op"] == "attn":
        state["q"] = normal(cu[-1], case["heads"], dim)
    return state


# ------------------------------------------------------------------ the plain forms
def _places(state):
    """Of each new token: its sequence, its number in it, its position, page and row of the page."""
    case = state["case"]
    n = torch.tensor(state["new"], device=DEV)
    seq = torch.repeat_interleave(torch.arange(len(state["new"]), device=DEV), n, output_size=state["cu"][-1])
    start = torch.tensor(state["cu"][:-1], device=DEV)
    at = torch.arange(state["cu"][-1], device=DEV) - start[seq]
    pos = state["kv_lens"].long()[seq] - n[seq] + at
    return seq, at, pos, state["table"].long()[seq, pos // case["page"]], pos % case["page"]


def _plain_read(state, places):
    page, row = places[3:]
    out = []
    for name in ("k", "v"):
        held, steps = _codes(state[name + "_pages"], state["case"]["dim"])
        out.append(_unpacked(held[page, :, row], steps[page, :, row], name == "k").to(torch.bfloat16))
    return tuple(out)


def _plain_append(state):
    places = _places(state)
    page, row = places[3:]
    for name in ("k", "v"):
        held, steps = _codes(state[name + "_pages"], state["case"]["dim"])
        code, byte = _quantised(state[name])
        held[page, :, row] = _packed(code, name == "k")
        steps[page, :, row] = byte
    return _plain_read(state, places)


def _plain_attn(state):
    case = state["case"]
    h, kv, dim = case["heads"], case["kv_heads"], case["dim"]
    seqs, most, longest = len(state["new"]), max(state["new"]), state["max_len"]
    seq, at = _places(state)[:2]
    q = torch.zeros(seqs, most, h, dim, device=DEV)
    q[seq, at] = state["q"].float()
    q = q.view(seqs, most, kv, h // kv, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv, h // kv * most, dim)
    table = state["table"].long().clamp(min=0)

    def cached(name):
        held, steps = _codes(state[name + "_pages"], dim)
        return _unpacked(held[table], steps[table], name == "k").transpose(2, 3).flatten(1, 2)[:, :longest].transpose(1, 2)

    score = (q @ cached("k").mT).mul_(dim ** -0.5)
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
    o = score.view(seqs, kv, h // kv * most, longest) @ cached("v")
    o = o.view(seqs, h, most, dim) / total
    return o.transpose(1, 2)[seq, at].to(state["q"].dtype), lse.transpose(1, 2)[seq, at].T.contiguous()


# ------------------------------------------------------------------ the framework's calls
def _own_rows(state):
    import mixed_length_dit_gb300 as zl
    if "batch" not in state:
        state["batch"] = zl.host_int32(state["cu"])
    cache = state["k_pages"], state["v_pages"], state["table"], state["kv_lens"], state["batch"]
    if state["case"]["op"] == "append":
        zl.paged_append_q4(state["k"], state["v"], *cache)
    return zl.paged_read_q4(*cache)


def _own_attn(state):
    import mixed_length_dit_gb300 as zl
    case = state["case"]
    if "batch" not in state:
        state["batch"] = zl.host_int32(state["cu"])
        state["workspace"] = zl.alloc_workspace(zl.paged_attn_q4_workspace_bytes(
            state["batch"], state["max_len"], case["heads"], case["kv_heads"], case["dim"], window=case["window"]), DEV)
    return zl.paged_attn_q4(state["q"], state["k_pages"], state["v_pages"], state["table"], state["kv_lens"],
                            state["batch"], state["max_len"], causal=case["causal"], window=case["window"],
                            workspace=state["workspace"])


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_attn(state) if op == "attn" else _own_rows(state)
    if op == "read":
        return _plain_read(state, _places(state))
    return _plain_append(state) if op == "append" else _plain_attn(state)


# ------------------------------------------------------------------ the definitions, in 64 bits
def _held(x):
    """The values that x [T, heads, d] is held as, group by group."""
    out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    for first in range(0, x.shape[-1], 32):
        g = x[..., first:first + 32].double()
        want = g.abs().amax(-1, keepdim=True) / 7
        unit = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -14))) - 3)      # of the last of four bits
        s = (torch.floor(want / unit + 0.5) * unit).clamp(max=61440)
        out[..., first:first + 32] = torch.where(s > 0, torch.floor(g / s + 0.5).clamp(-8, 7) * s, 0.0)
    return out


def _values(pool, numbers, head, dim, keys):
    """The values [tokens, d] behind pages `numbers` of one head, byte by byte."""
    page = pool.shape[2]
    block = pool[numbers, head].flatten(1)
    held = block[:, :page * dim // 2].reshape(-1, dim // 2).int()
    byte = block[:, page * dim // 2:].reshape(-1, dim // 32).long()
    e, m = byte >> 3, (byte & 7).double()
    s = torch.where(e > 0, (1 + m / 8) * ((e - 15 + 1023) << 52).view(torch.float64), m / 8 * 2.0 ** -14)
    out = torch.empty(held.shape[0], dim, dtype=torch.float64, device=DEV)
    groups = dim // 32
    for j in range(dim):
        group, i = divmod(j, 32)
        if keys:        # word i / 8 of the group: piece i / 8, in it word `group`
            at = (i // 8 * groups + group) * 4 + i % 8 // 2
        else:
            at = (i // 4 * groups + group) * 2 + i % 4 // 2
        out[:, j] = ((held[:, at] >> 4 * (i % 2) & 15) - 8).double() * s[:, group]
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "append":
        return _held(state["k"]), _held(state["v"])
    new, lens, cu, page, dim = state["new"], state["lens"], state["cu"], case["page"], case["dim"]
    if case["op"] == "read":
        out = []
        for name in ("k", "v"):
            x = torch.empty(cu[-1], case["kv_heads"], dim, dtype=torch.float64, device=DEV)
            for s, n in enumerate(lens):
                for g in range(case["kv_heads"]):
                    numbers = state["table"][s, :-(-n // page)].long()
                    x[cu[s]:cu[s + 1], g] = _values(state[name + "_pages"], numbers, g, dim, name == "k")[:n]
            out.append(x)
        return tuple(out)
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
            k, v = (_values(state[x + "_pages"], numbers, g, dim, x == "k")[:b] for x in ("k", "v"))
            for i in range(g * group, (g + 1) * group):
                x = state["q"][cu[s]:cu[s + 1], i].double() @ k.T / math.sqrt(dim)
                x[hidden] = -math.inf
                lse[i, cu[s]:cu[s + 1]] = torch.logsumexp(x, 1)
                out[cu[s]:cu[s + 1], i] = torch.softmax(x, 1) @ v
    return out, lse
