"""What the attention layers of a block-diffusion Mamba hybrid need beside attention itself, as
cases to be timed: rotary positions of queries and keys (alone, or on the way into the pages),
attention whose scores are capped, biased by distance or masked by document and prefix, and the
upkeep of a paged cache (a block's pages taken and the window's given back, streams forked, a
pool compacted, pages copied).

`listed()` names the cases, `draw()` gives others of the same ranges, `prepare()` makes a case's
inputs on the GPU, `run()` makes one pass (the plain form in elementary torch operations, or
the library's calls where `own` is set), `work()` counts the bytes and operations that a pass
cannot do without, `exact()` is the operator's definition in 64 bits.

Head counts and lengths are those of the workload shapes in configs.py (24, 16 and 40 attention
heads of 64 for the 700M, 350M and 3B shapes; blocks of 32 tokens, running sets of 128, prefixes
of 8K to 256K) or generic ones.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
PLAIN, LINEAR, BASE, PARTS = range(4)  # how rotary frequencies are scaled
LOW, HIGH, TRAINED = 1.0, 32.0, 8192   # PARTS: turns within the trained length


# ------------------------------------------------------------------------------------- cases
def _rotary(name, **kw):
    c = dict(name=name, op="rotary", append=False, batch=1, tokens=32, prefix=8192, heads=24, kv_heads=4, headdim=64,
             dtype="bf16", page=32, ragged=False, dim=64, interleaved=False, kind=PLAIN, factor=1.0)
    c.update(kw)
    return c


def _attn(name, **kw):
    c = dict(name=name, op="attn", batch=1, tokens=32, prefix=8192, heads=24, kv_heads=4, headdim=64, dtype="bf16",
             page=32, ragged=False, block=0, window=0, sinks=0, cap=0.0, bias=False, documents=0, prefix_mask=False)
    c.update(kw)
    return c


def _pages(name, op, **kw):
    c = dict(name=name, op=op, batch=4, tokens=32, prefix=2000, page=32, spare=1.5)
    if op == "advance":
        c.update(window=0, sinks=0, ragged=False)
    else:
        c.update(kv_heads=4, headdim=64, dtype="bf16", layers=1)
    c.update(kw)
    return c


def listed():
    return [
        # a denoising step's block of the 3B shape far into its context: all latency
        _rotary("rotary_block", prefix=262144, heads=40, kv_heads=8),
        # prompts of unequal lengths on their way into the pages, three quarters of a head
        # rotated, frequencies scaled by parts
        _rotary("rotary_prompts", append=True, batch=4, tokens=16384, prefix=1000, heads=20, headdim=128, page=64,
                ragged=True, dim=96, interleaved=True, kind=PARTS, factor=8.0),
        # one token of each of 16 streams, capped scores: a decode step of a capped model
        _attn("capped_token", batch=16, tokens=1, prefix=4000, heads=16, kv_heads=8, page=64, ragged=True, cap=50.0),
        # a prompt's second chunk in block order, capped, heads of 128
        _attn("capped_prompt", tokens=8192, prefix=8192, heads=20, headdim=128, page=128, block=32, cap=30.0),
        # denoising of 64 streams, running sets of 4 x 32, scores biased by distance
        _attn("biased_running_set", batch=64, tokens=128, prefix=32768, page=64, ragged=True, bias=True),
        # documents of some 700 tokens packed into one causal float32 prompt behind a short cache, with
        # a cap, a bias and padding at the end that attends to nothing
        _attn("documents_f32", tokens=8191, prefix=77, heads=16, kv_heads=4, page=16, dtype="f32", block=1, cap=20.0,
              bias=True, documents=700),
        # one prompt forked into four samples, one layer
        _pages("fork_sample", "fork", prefix=1000),
        # beams of a running set: 64 streams from 16 parents, eight layers
        _pages("fork_beams", "fork", batch=64, prefix=16384, page=64, layers=8),
        # the next block's pages of four streams
        _pages("advance_block", "advance"),
        # 64 long streams with a sliding window on short pages
        _pages("advance_window", "advance", batch=64, tokens=128, prefix=262144, page=16, window=4096, sinks=4,
               ragged=True, spare=1.1),
        # pools after streams have ended: a small one, and one of two layers with many moves
        _pages("compact_small", "compact", batch=8, prefix=1000, page=16),
        _pages("compact_pool", "compact", batch=32, prefix=8192, page=128, layers=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "attn", "attn", "attn", "fork", "advance", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128, 256])
    ragged = rng.random() < 0.5
    D = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 3, 4, 5, 8])
    if op == "rotary":
        c = _rotary("", append=rng.random() < 0.5, batch=_log(rng, 1, 64), tokens=_log(rng, 1, 16384),
                    prefix=_log(rng, 1, 262144), heads=heads, kv_heads=kv, headdim=D, dtype=dtype, page=page, ragged=ragged,
                    dim=rng.choice([D, D, D // 2, 3 * D // 4, 2 * rng.randint(1, D // 2)]), interleaved=rng.random() < 0.5,
                    kind=rng.choice([PLAIN, LINEAR, BASE, PARTS]), factor=rng.choice([2.0, 4.0, 32.0]))
        if c["append"]:  # a pool of pages comes with it
            c["prefix"] = min(c["prefix"], 16384)
            while c["batch"] * kv * (c["prefix"] + c["tokens"]) * D > 6e7:
                c["batch"] = max(1, c["batch"] // 2)
                c["tokens"] = max(1, c["tokens"] // 2)
        while c["batch"] * c["tokens"] * heads * D * (1 if dtype == "bf16" else 2) > 1.6e8:
            c["tokens"] = max(1, c["tokens"] // 2)
        if c["kind"] == BASE and c["dim"] == 2:
            c["kind"] = LINEAR
        del c["name"]
        return c
    if op == "attn":
        window = _log(rng, 1, 8192) if rng.random() < 0.25 else 0
        c = _attn("", batch=_log(rng, 1, 64), tokens=_log(rng, 1, 4096), prefix=_log(rng, 1, 65536), heads=heads, kv_heads=kv,
                  headdim=D, dtype=dtype, page=page, ragged=ragged, block=rng.choice([0, 1, 32]), window=window,
                  sinks=rng.choice([0, 4, 33]) if window else 0, cap=rng.choice([0.0, 5.0, 30.0, 50.0]),
                  bias=rng.random() < 0.5, documents=_log(rng, 8, 4096) if rng.random() < 0.3 else 0,
                  prefix_mask=rng.random() < 0.3)
        while c["batch"] * heads * c["tokens"] * (c["prefix"] + c["tokens"]) > (1.9e9 if dtype == "bf16" else 2e8):
            c["tokens" if c["tokens"] > 128 else "prefix" if c["prefix"] > 4096 else "batch" if c["batch"] > 1 else "prefix"] //= 2
        while c["batch"] * kv * (c["prefix"] + c["tokens"]) * D > 2.5e8:
            c["prefix"] //= 2
        del c["name"]
        return c
    if op == "advance":
        window = _log(rng, 1, 8192) if rng.random() < 0.5 else 0
        c = _pages("", op, batch=_log(rng, 1, 256), tokens=_log(rng, 1, 1024), prefix=_log(rng, 1, 262144), page=page,
                   window=window, sinks=rng.choice([0, 4, 33]) if window else 0, ragged=ragged,
                   spare=rng.choice([0.5, 1.02, 1.5]))
        while c["batch"] * (c["prefix"] + c["tokens"]) / page > 1.1e6:
            c["prefix"] //= 2
        del c["name"]
        return c
    c = _pages("", op, batch=_log(rng, 1, 64), prefix=_log(rng, 1, 16384), page=page, kv_heads=kv, headdim=D, dtype=dtype,
               layers=rng.choice([1, 2, 4, 8]), spare=rng.choice([0.5, 1.5]))
    while c["batch"] * kv * (c["prefix"] + 2 * page) * D * c["layers"] > 1.1e8:
        c["layers" if c["layers"] > 1 else "prefix" if c["prefix"] > 64 else "batch"] //= 2
    del c["name"]
    return c


# ------------------------------------------------------------------- lengths (from the case)
def _counts(c):
    """New tokens of each stream: `tokens`, or where ragged down to half of it (one of several
    streams has none)."""
    T, n = c["tokens"], c["batch"]
    if not c["ragged"]:
        return [T] * n
    return [0 if i == 1 and n > 2 else T - (i * 7919 + 13) % (T // 2 + 1) for i in range(n)]


def _lens(c):
    """Cached tokens of each stream: `prefix`, or where ragged (or the pool is forked or
    compacted) down to half of it."""
    L, n = c["prefix"], c["batch"]
    if not c.get("ragged", True):
        return [L] * n
    return [L - (i * 6271) % (L // 2 + 1) for i in range(n)]


def _documents(c, end):
    """Borders of the documents in a stream's positions [0, end)."""
    borders, i = [0], 0
    while borders[-1] < end:
        borders.append(borders[-1] + max(1, c["documents"] * (500 + i * 7919 % 1000) // 1000))
        i += 1
    return borders


def _ranges(c, n, length):
    """(first, last) key of each of a stream's new tokens: its document's; the last 64th of the
    tokens is padding, which attends to nothing."""
    b = _documents(c, length + n + 1)
    first, last, d = [], [], 0
    for i in range(n):
        while b[d + 1] <= length + i:
            d += 1
        pad = i >= n - n // 64
        first.append(0 if pad else b[d])
        last.append(0 if pad else b[d + 1])
    return first, last


def _visible(c, n, length):
    """(query, key) pairs that the mask leaves of a stream with n new tokens after `length`
    cached ones, and how many different keys they touch."""
    blk, win, sinks, end = c["block"], c["window"], c["sinks"], length + n
    pref = length + n // 3 if c["prefix_mask"] else 0
    first, last = _ranges(c, n, length) if c["documents"] else ([0] * n, [end] * n)
    pairs, touched = 0, np.zeros(end + 1, dtype=np.int64)
    for p in range(length, end):
        f = first[p - length]
        hi = min(end, last[p - length], max((p // blk + 1) * blk, pref) if blk else end)
        lo = max(f, p - win + 1 if win else 0)
        for a, b in ((lo, hi), (f, min(hi, sinks, lo) if win else 0)):
            if a < b:
                pairs += b - a
                touched[a] += 1
                touched[b] -= 1
    return pairs, int((np.cumsum(touched) > 0).sum())


def _elt(c):
    return 2 if c["dtype"] == "bf16" else 4


def work(c):
    if c["op"] == "rotary":
        n, e = sum(_counts(c)), _elt(c)
        kv = c["kv_heads"] * (2 if c["append"] else 1)
        return {"bytes": 2 * n * (c["heads"] + kv) * c["headdim"] * e, "flops": 3 * n * (c["heads"] + c["kv_heads"]) * c["dim"]}
    if c["op"] == "attn":
        e, pairs, keys = _elt(c), 0, 0
        for n, length in zip(_counts(c), _lens(c)):
            p, k = _visible(c, n, length)
            pairs, keys = pairs + p, keys + k
        io = 2 * sum(_counts(c)) * c["heads"] * c["headdim"] * e  # queries and outputs
        return {"bytes": io + 2 * keys * c["kv_heads"] * c["headdim"] * e,
                "flops": 4 * pairs * c["heads"] * c["headdim"]}
    entries = 8 * c["batch"] * _per(c) + 8 * _pool(c)  # table and uses, in and out
    if c["op"] == "advance":
        return {"bytes": entries, "flops": 0}
    page = c["kv_heads"] * c["page"] * c["headdim"] * _elt(c)
    if c["op"] == "fork":
        parents, lens = _parents(c), _lens(c)
        moved = sum(p in parents[:b] and lens[p] % c["page"] > 0 for b, p in enumerate(parents) if p >= 0)
    else:
        live = _live(c)
        moved = int(live * (1 - live / _pool(c)))  # of pages that lie anywhere in the pool
    return {"bytes": entries + 4 * moved * page * c["layers"], "flops": 0}


# ------------------------------------------------------------------------------------ inputs
def _per(c):
    """Entries of a table row."""
    return -(-(c["prefix"] + c["tokens"]) // c["page"])


def _held(c):
    """Pages of each stream."""
    return [-(-n // c["page"]) for n in _lens(c)]


def _pool(c):
    if c["op"] == "compact":
        return 3 + sum(_held(c))
    if c["op"] == "fork":
        return 3 + sum(_held(c)) + int(c["batch"] * c["spare"])
    lens, n = _lens(c), 0  # advance: what the streams hold, and `spare` of what they need
    need = sum(max(0, -(-min(L + t, _per(c) * c["page"]) // c["page"]) - -(-L // c["page"])) for L, t in zip(lens, _counts(c)))
    for L in lens:
        n += -(-L // c["page"]) - _gone(c, L)
    return n + int(need * c["spare"]) + 1


def _gone(c, length):
    """Pages of a stream that an earlier call has given back: those a block earlier that the
    window had left."""
    if not c["window"]:
        return 0
    at = length - c["tokens"] - c["window"] + 1
    return max(0, at // c["page"] - -(-c["sinks"] // c["page"]))


def _parents(c):
    """Streams forked: each fourth one into itself and its three neighbours; of several such
    groups the last ends instead."""
    p = [b // 4 * 4 for b in range(c["batch"])]
    if c["batch"] > 8:
        p[-2:] = [-1, -1]
    return p


def _ended(c):
    """Streams of the pool to be compacted whose pages were given back: every third one."""
    return [b for b in range(c["batch"]) if b % 3 == 1]


def _live(c):
    held = _held(c)
    return sum(n for b, n in enumerate(held) if b not in _ended(c))


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(c):
    n = _counts(c)
    return _ints([sum(n[:i]) for i in range(len(n) + 1)]) if c["ragged"] else None


def _chunk(c, g, scale):
    """Queries, keys and values: slices of one projection's rows."""
    dt, D, kv, H, n = DTYPES[c["dtype"]], c["headdim"], c["kv_heads"], c["heads"], sum(_counts(c))
    qkv = _randn(g, (n, (H + 2 * kv) * D), dt)
    qkv[:, : H * D] *= scale
    return {"q": qkv[:, : H * D].view(n, H, D), "k": qkv[:, H * D : (H + kv) * D].view(n, kv, D),
            "v": qkv[:, (H + kv) * D :].view(n, kv, D), "n": n, "starts": _starts(c), "lens": _ints(_lens(c))}


def _cache(c, g):
    """A pool of pages in random order with each stream's table. Under a window the pages that
    no query will see again have been given back: their entries are -1."""
    dt, page, D = DTYPES[c["dtype"]], c["page"], c["headdim"]
    per = _per(c)
    pool = c["batch"] * per + 3
    shape = (pool, c["kv_heads"], page, D)
    k, v = _randn(g, shape, dt), _randn(g, shape, dt)
    table = torch.randperm(pool, generator=g, device="cuda")[: c["batch"] * per].to(torch.int32).reshape(c["batch"], per)
    if c.get("window"):
        first = torch.arange(per, device="cuda") * page
        gone = (first[None] >= c["sinks"]) & (first[None] + page <= _ints(_lens(c))[:, None] - c["window"] + 1)
        table = torch.where(gone, torch.full_like(table, -1), table)
    return {"k_pages": k, "v_pages": v, "table": table}


def prepare(c, seed):
    g = _gen(seed)
    s = {"case": c}
    if c["op"] == "rotary":
        s.update(_chunk(c, g, 1.0), lens_out=torch.empty(c["batch"], dtype=torch.int32, device="cuda"))
        s.update(q_out=torch.empty((s["n"], c["heads"], c["headdim"]), dtype=s["q"].dtype, device="cuda"),
                 k_out=torch.empty((s["n"], c["kv_heads"], c["headdim"]), dtype=s["q"].dtype, device="cuda"))
        if c["append"]:
            s.update(_cache(c, g))
        s["freqs"] = torch.from_numpy(_frequencies(c)).cuda()
    elif c["op"] == "attn":
        s.update(_chunk(c, g, 2.0), **_cache(c, g))
        s["out"] = torch.empty((s["n"], c["heads"], c["headdim"]), dtype=s["q"].dtype, device="cuda")
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["heads"] + 1, device="cuda") / c["heads"]) if c["bias"] else None
        s["first"] = s["last"] = s["prefix"] = None
        if c["documents"]:
            r = [_ranges(c, n, length) for n, length in zip(_counts(c), _lens(c))]
            s["first"], s["last"] = (_ints([x for f in r for x in f[i]]) for i in (0, 1))
        if c["prefix_mask"]:
            s["prefix"] = _ints([length + n // 3 for n, length in zip(_counts(c), _lens(c))])
    else:
        _prepare_pages(c, g, s)
    if own:
        _plan(s)
    return s


def _prepare_pages(c, g, s):
    """A pool that streams share out among themselves: each holds pages from anywhere in it."""
    P, per, held = _pool(c), _per(c), _held(c)
    order = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    ended = _ended(c) if c["op"] == "compact" else []
    used = torch.zeros((c["batch"], per), dtype=torch.bool)
    for b, L in enumerate(_lens(c)):
        if b not in ended:
            used[b, : held[b]] = True
            if c["op"] == "advance" and c["window"]:
                at = -(-c["sinks"] // c["page"])
                used[b, at : at + _gone(c, L)] = False
    used = used.cuda()
    rank = torch.cumsum(used.view(-1).long(), 0).view(c["batch"], per) - 1
    table = torch.where(used, order[rank.clamp(min=0)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    uses = torch.zeros(P + 1, dtype=torch.int32, device="cuda")
    uses[torch.where(used, table, P).long().view(-1)] = 1
    lens = _lens(c)
    s.update(table=table, uses=uses[:P].clone(), table_out=torch.empty_like(table), uses_out=torch.empty_like(uses[:P]),
             lens=_ints([0 if b in ended else n for b, n in enumerate(lens)]), lens_out=torch.empty_like(_ints(lens)),
             count=torch.empty(1, dtype=torch.int32, device="cuda"))
    if c["op"] == "advance":
        s.update(starts=_starts(c))
        return
    shape = (P, c["kv_heads"], c["page"], c["headdim"])
    s["pools"] = [(_randn(g, shape, DTYPES[c["dtype"]]), _randn(g, shape, DTYPES[c["dtype"]])) for _ in range(c["layers"])]
    s["copies"] = torch.empty((c["batch"] if c["op"] == "fork" else P // 2, 2), dtype=torch.int32, device="cuda")
    if c["op"] == "fork":
        s["parents"] = _ints(_parents(c))


def _frequencies(c, t=np.float64):
    """Radians per position of each rotated pair."""
    dim, s = c["dim"], t(c["factor"])
    base = t(10000) * (s ** (t(dim) / t(dim - 2)) if c["kind"] == BASE else t(1))
    f = base ** (-2 * np.arange(dim // 2, dtype=t) / t(dim))
    if c["kind"] == LINEAR:
        f = f / s
    if c["kind"] == PARTS:
        g = np.clip((TRAINED * f / (2 * np.pi) - LOW) / (HIGH - LOW), 0, 1)
        f = f * (g + (1 - g) / s)
    return f


def _plan(s):
    """What a program of the library keeps beside its tensors: descriptors and workspaces."""
    from bidirectional_mamba_state_amd import bdssm
    c = s["case"]
    space = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda") if n else None  # noqa: E731
    if c["op"] in ("rotary", "attn"):
        dt = bdssm.BF16 if c["dtype"] == "bf16" else bdssm.F32
        s["dims"] = bdssm.attn_dims(c["batch"], c["heads"], c["kv_heads"], c["headdim"], dt, c["page"])
        if "table" in s:
            s["cache"] = bdssm.KvCache(s["dims"], s["k_pages"], s["v_pages"], s["table"], s["lens"], c["prefix"])
    if c["op"] == "rotary":
        s["turns"] = bdssm.rotary_turns(c["dim"], base=10000.0, factor=c["factor"], trained=TRAINED, low=LOW, high=HIGH,
                                        kind=(bdssm.ROTARY_PLAIN, bdssm.ROTARY_LINEAR, bdssm.ROTARY_BASE,
                                              bdssm.ROTARY_PARTS)[c["kind"]])
        s["rotary"] = bdssm.Rotary(s["turns"], interleaved=c["interleaved"])
    elif c["op"] == "attn":
        s["mask"] = bdssm.attn_mask(c["headdim"] ** -0.5, c["block"], c["window"], c["sinks"])
        s["scores"] = bdssm.AttnScores(cap=c["cap"], slopes=s["slopes"], prefix=s["prefix"], first=s["first"], last=s["last"])
        s["ws"] = space(bdssm.attn_step_ex_workspace(s["dims"], c["tokens"], c["prefix"], s["mask"], s["scores"]))
    else:
        s["pd"] = bdssm.page_dims(c["batch"], c["page"], s["uses"].numel(), s["table"].shape[1])
        s["pages"] = bdssm.Pages(s["pd"], s["table"], s["lens"], s["uses"])
        s["ws"] = space(bdssm.pages_workspace(s["pd"]))
        if c["op"] != "advance":
            dt = bdssm.BF16 if c["dtype"] == "bf16" else bdssm.F32
            s["dims"] = bdssm.attn_dims(c["batch"], c["kv_heads"], c["kv_heads"], c["headdim"], dt, c["page"])
            s["caches"] = [bdssm.KvCache(s["dims"], k, v, s["table_out"], s["lens"], c["prefix"]) for k, v in s["pools"]]


# -------------------------------------------------------------------------------------- runs
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from bidirectional_mamba_state_amd import bdssm
    c = s["case"]
    if c["op"] == "rotary":
        if c["append"]:
            bdssm.rotary_append(s["dims"], c["tokens"], s["rotary"], s["q"], s["k"], s["v"], s["cache"], s["q_out"],
                                lens_out=s["lens_out"], starts=s["starts"])
            return s["q_out"], s["k_pages"], s["v_pages"], s["lens_out"]
        bdssm.rotary_step(s["dims"], c["tokens"], s["rotary"], s["q"], s["k"], s["q_out"], s["k_out"], lens=s["lens"],
                          starts=s["starts"])
        return s["q_out"], s["k_out"]
    if c["op"] == "attn":
        bdssm.attn_step_ex(s["dims"], c["tokens"], s["q"], s["k"], s["v"], s["cache"], s["mask"], s["scores"], s["out"],
                           s["ws"], starts=s["starts"])
        return s["out"]
    if c["op"] == "advance":
        bdssm.pages_advance(s["pd"], s["pages"], c["tokens"], s["table_out"], s["uses_out"], s["count"], s["ws"],
                            window=c["window"], sinks=c["sinks"], starts=s["starts"])
        return s["table_out"], s["uses_out"], s["count"]
    if c["op"] == "fork":
        bdssm.pages_fork(s["pd"], s["pages"], s["parents"], s["table_out"], s["lens_out"], s["uses_out"], s["copies"],
                         s["count"], s["ws"])
    else:
        bdssm.pages_compact(s["pd"], s["pages"], s["table_out"], s["uses_out"], s["copies"], s["count"], s["ws"])
    for cache in s["caches"]:
        bdssm.pages_copy(s["dims"], cache, s["copies"])
    return _pages_out(s)


def _pages_out(s):
    out = [s["table_out"], s["uses_out"], s["copies"], s["count"]]
    if s["case"]["op"] == "fork":
        out.append(s["lens_out"])
    return out + [p for pools in s["pools"] for p in pools]


def _run_plain(s):
    return {"rotary": _plain_rotary, "attn": _plain_attn, "advance": _plain_advance, "fork": _plain_fork,
            "compact": _plain_compact}[s["case"]["op"]](s)


def _of_token(s):
    """Stream of each new token, and its place there."""
    c = s["case"]
    tok = torch.arange(s["n"], device=s["q"].device)
    if s["starts"] is None:
        of, st = tok // c["tokens"], torch.arange(c["batch"] + 1, device=tok.device) * c["tokens"]
    else:
        st = s["starts"].long()
        of = torch.searchsorted(st[1:].contiguous(), tok, right=True)
    return of, tok - st[of], st


def _plain_rotary(s):
    c = s["case"]
    of, i, st = _of_token(s)
    pos = s["lens"].long()[of] + i
    angle = pos.double()[:, None] * s["freqs"][None]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x, out):
        x, h = x.float(), c["dim"] // 2
        if c["interleaved"]:
            a, b = x[..., : c["dim"] : 2], x[..., 1 : c["dim"] : 2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = x[..., :h], x[..., h : 2 * h]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        return torch.cat([y, x[..., c["dim"] :]], -1).to(out)

    q, k = turned(s["q"], s["q"].dtype), turned(s["k"], s["q"].dtype)
    if not c["append"]:
        return q, k
    page, slot = s["table"].long()[of, pos // c["page"]], pos % c["page"]
    s["k_pages"][page, :, slot] = k
    s["v_pages"][page, :, slot] = s["v"]
    torch.add(s["lens"], (st[1:] - st[:-1]).to(torch.int32), out=s["lens_out"])
    return q, s["k_pages"], s["v_pages"], s["lens_out"]


def _plain_attn(s):
    c = s["case"]
    b, T, L, H, kv, D = c["batch"], c["tokens"], c["prefix"], c["heads"], c["kv_heads"], c["headdim"]
    G, dev = H // kv, s["q"].device
    step = torch.arange(T, device=dev)
    if s["starts"] is None:
        rows, new = (torch.arange(b, device=dev) * T)[:, None] + step[None], torch.ones((b, T), dtype=torch.bool, device=dev)
    else:
        st = s["starts"].long()
        rows, new = st[:-1, None] + step[None], step[None] < (st[1:] - st[:-1])[:, None]
        rows = rows.clamp(max=max(0, s["n"] - 1))
    # keys and values of every stream: its cached tokens, then the chunk's own
    npg = -(-L // c["page"])
    table = s["table"][:, :npg].long()
    at = torch.arange(L, device=dev)
    there = (at[None] < s["lens"][:, None]) & (table >= 0).repeat_interleave(c["page"], dim=1)[:, :L]
    ok = torch.cat([there, new], 1)
    pos = torch.cat([at[None].expand(b, L), s["lens"][:, None] + step[None]], 1)

    def keys(pages, fresh):
        old = pages[table.clamp(min=0)].permute(0, 2, 1, 3, 4).reshape(b, kv, npg * c["page"], D)[:, :, :L]
        return torch.cat([old.float(), fresh[rows].permute(0, 2, 1, 3).float()], 2)

    qpos = s["lens"][:, None] + step[None]
    see = ok[:, None, :].expand(b, T, L + T)
    if c["block"]:
        in_order = pos[:, None] // c["block"] <= qpos[:, :, None] // c["block"]
        if s["prefix"] is not None:
            in_order |= pos[:, None] < s["prefix"][:, None, None]
        see = see & in_order
    if c["window"]:
        see = see & ((qpos[:, :, None] - pos[:, None] < c["window"]) | (pos[:, None] < c["sinks"]))
    if s["first"] is not None:
        see = see & (pos[:, None] >= s["first"][rows][:, :, None]) & (pos[:, None] < s["last"][rows][:, :, None])
    q = s["q"][rows].float().view(b, T, kv, G, D).permute(0, 2, 3, 1, 4).reshape(b, kv, G * T, D)
    p = torch.matmul(q * D ** -0.5, keys(s["k_pages"], s["k"]).transpose(2, 3).contiguous()).view(b, kv, G, T, L + T)
    if c["cap"]:
        p.div_(c["cap"]).tanh_().mul_(c["cap"])
    if c["bias"]:
        far = (qpos[:, :, None] - pos[:, None]).abs_().float()
        p.addcmul_(s["slopes"].view(1, kv, G, 1, 1), far[:, None, None], value=-1.0)
        del far
    p.masked_fill_(~see[:, None, None], float("-inf"))
    p.sub_(p.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, kv, G * T, L + T), keys(s["v_pages"], s["v"]).masked_fill_(~ok[:, None, :, None], 0.0))
    o = o.view(b, kv, G, T, D) / total.masked_fill_(total == 0, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(b * T, H, D).to(s["q"].dtype)
    if s["starts"] is None:
        return o
    of, i, _ = _of_token(s)  # back to the tokens' own order
    return o[of * T + i]


def _lowest_free(uses, most):
    """The free pages, ascending, then -1 (`most` of them)."""
    free = uses <= 0
    P = uses.numel()
    page = torch.full((max(P, most) + 1,), -1, dtype=torch.int32, device=uses.device)
    page.scatter_(0, torch.where(free, torch.cumsum(free.long(), 0) - 1, max(P, most)),
                  torch.arange(P, dtype=torch.int32, device=uses.device))
    page[-1:] = -1
    return page[:most], free.sum()


def _counted(table, P):
    """How many entries name each page."""
    n = torch.zeros(P + 1, dtype=torch.int32, device=table.device)
    return n.scatter_add_(0, torch.where(table >= 0, table, P).long().view(-1), torch.ones_like(table).view(-1))[:P]


def _plain_advance(s):
    c = s["case"]
    page, table, lens = c["page"], s["table"], s["lens"].long()
    per = table.shape[1]
    n = torch.full_like(lens, c["tokens"]) if s["starts"] is None else (s["starts"][1:] - s["starts"][:-1]).long()
    end = (lens + n).clamp(max=per * page)
    at = torch.arange(per, device=table.device)[None] * page
    needed = at < end[:, None]
    if c["window"]:
        needed &= (at < c["sinks"]) | (at + page > lens[:, None] - c["window"] + 1)
    lacks = needed & (table < 0) & (at >= lens[:, None])
    rank = torch.cumsum(lacks.view(-1).long(), 0).view_as(table) - 1
    fresh, free = _lowest_free(s["uses"], table.numel())
    kept = torch.where(needed, table, torch.full_like(table, -1))
    out = torch.where(lacks, fresh[rank.clamp(min=0)], kept)
    uses = s["uses"] + _counted(out, s["uses"].numel()) - _counted(table, s["uses"].numel())
    return out, uses, (lacks.sum() - free).clamp(min=0).to(torch.int32).view(1)


def _copied(s, copies):
    """The pages of the list copied in every layer's pools; a row of -1 repeats one that is none
    (or copies a page to itself)."""
    some = copies[(copies[:, :1] >= 0).long().argmax(0)].clamp(min=0) if len(copies) else copies
    rows = torch.where(copies >= 0, copies, some).long()
    for pools in s["pools"]:
        for p in pools:
            p[rows[:, 1]] = p[rows[:, 0]]


def _plain_fork(s):
    c = s["case"]
    page, table, par = c["page"], s["table"], s["parents"].long()
    per, P = table.shape[1], s["uses"].numel()
    own_ = par >= 0
    p = par.clamp(min=0)
    lens = torch.where(own_, s["lens"][p], 0)
    again = ((par[:, None] == par[None]) & torch.ones_like(par[:, None] * par[None]).tril(-1).bool()).any(1)
    rows = torch.where(own_[:, None], table[p], -1)
    at = torch.arange(per, device=table.device)[None]
    full, part = (lens // page)[:, None], (lens % page > 0)[:, None]
    here = (at == full) & part & again[:, None]
    old = torch.where(here, rows, -1).amax(1)
    needs = old >= 0
    fresh, free = _lowest_free(s["uses"], c["batch"])
    new = torch.where(needs, fresh[(torch.cumsum(needs.long(), 0) - 1).clamp(min=0)], -1)
    out = torch.where(again[:, None] & (at >= full), torch.where(here, new[:, None], -1), rows)
    uses = s["uses"] + _counted(out, P) - _counted(table, P)
    done = (needs & (new >= 0))[:, None]
    copies = torch.where(done, torch.stack([old, new], 1), -1)
    _copied(s, copies)
    return [out, uses, copies, (needs.sum() - free).clamp(min=0).to(torch.int32).view(1), lens] + [
        x for pools in s["pools"] for x in pools]


def _plain_compact(s):
    table, uses = s["table"], s["uses"]
    P = uses.numel()
    idx = torch.arange(P, dtype=torch.int32, device=uses.device)
    on = uses > 0
    live = on.sum()
    below = torch.cumsum(on.long(), 0) - on.long()  # live pages in front
    low = ~on & (idx < live)
    high = on & (idx >= live)
    dump = P // 2
    free = torch.full((dump + 1,), -1, dtype=torch.int32, device=uses.device)
    free.scatter_(0, torch.where(low, idx - below, dump), idx)
    src = torch.full((dump + 1,), -1, dtype=torch.int32, device=uses.device)
    src.scatter_(0, torch.where(high, live - 1 - below, dump), idx)  # the highest first
    copies = torch.stack([src[:dump], free[:dump]], 1)
    to = torch.where(high, free[torch.where(high, live - 1 - below, dump)], idx)
    out = torch.where(table >= 0, to[table.clamp(min=0).long()], table)
    moved = torch.zeros_like(uses).scatter_add_(0, to.long(), torch.where(on, uses, 0))
    _copied(s, copies)
    return [out, moved, copies, live.to(torch.int32).view(1)] + [x for pools in s["pools"] for x in pools]


# ------------------------------------------------------------------------------------- exact
def exact(c, seed):
    s = prepare(c, seed)
    return {"rotary": _exact_rotary, "attn": _exact_attn, "advance": _exact_advance, "fork": _exact_fork,
            "compact": _exact_compact}[c["op"]](c, s)


def _exact_rotary(c, s):
    pos = np.concatenate([np.arange(length, length + n) for n, length in zip(_counts(c), _lens(c))] + [np.zeros(0, int)])
    f = _frequencies(c, np.longdouble)
    angle = np.mod(pos.astype(np.longdouble)[:, None] * f[None], 2 * np.longdouble(np.pi))
    turn = torch.from_numpy(np.exp(1j * angle.astype(np.float64))).cuda()[:, None]

    def turned(x):
        x = x.double()
        y = x.clone()
        pair = (slice(0, c["dim"], 2), slice(1, c["dim"], 2)) if c["interleaved"] else \
            (slice(0, c["dim"] // 2), slice(c["dim"] // 2, c["dim"]))
        z = torch.complex(x[..., pair[0]], x[..., pair[1]]) * turn
        y[..., pair[0]], y[..., pair[1]] = z.real, z.imag
        return y

    q, k = turned(s["q"]), turned(s["k"])
    if not c["append"]:
        return q, k
    kp, vp, first, table = s["k_pages"].double(), s["v_pages"].double(), 0, s["table"].tolist()
    lens = _lens(c)
    for b, n in enumerate(_counts(c)):
        t = 0
        while t < n:  # a page's worth of tokens at a time
            page, slot = divmod(lens[b] + t, c["page"])
            m = min(n - t, c["page"] - slot)
            for pages, new in ((kp, k), (vp, s["v"])):
                pages[table[b][page], :, slot : slot + m] = new[first + t : first + t + m].transpose(0, 1).double()
            t += m
        first += n
    return q, kp, vp, _ints([a + b for a, b in zip(lens, _counts(c))])


def _exact_attn(c, s):
    page, D, kv, G, first = c["page"], c["headdim"], c["kv_heads"], c["heads"] // c["kv_heads"], 0
    out = torch.zeros((s["n"], c["heads"], D), dtype=torch.float64, device="cuda")
    for b, (n, length) in enumerate(zip(_counts(c), _lens(c))):
        used = -(-length // page)
        ids = s["table"][b, :used].long()
        j = torch.arange(length + n, device="cuda")
        p = torch.arange(length, length + n, device="cuda")[:, None]
        held = torch.cat([(ids >= 0).repeat_interleave(page)[:length], torch.ones(n, dtype=torch.bool, device="cuda")])
        see = held[None].expand(n, -1)
        if c["block"]:
            last = (p // c["block"] + 1) * c["block"]
            see = see & (j[None] < (last.clamp(min=length + n // 3) if c["prefix_mask"] else last))
        if c["window"]:
            see = see & ((j[None] > p - c["window"]) | (j[None] < c["sinks"]))
        if c["documents"]:
            lo, hi = (torch.tensor(x, device="cuda").view(-1, 1) for x in _ranges(c, n, length))
            see = see & (j[None] >= lo) & (j[None] < hi)
        for h in range(kv if n else 0):
            K, V = (torch.cat([pages[ids.clamp(min=0), h].reshape(-1, D)[:length].double(),
                               new[first : first + n, h].double()]) for pages, new in ((s["k_pages"], s["k"]), (s["v_pages"], s["v"])))
            for t0 in range(0, n, 1024):
                t1 = min(n, t0 + 1024)
                q = s["q"][first + t0 : first + t1, h * G : (h + 1) * G].double()
                sc = (q.reshape(-1, D) @ K.t()).reshape(t1 - t0, G, -1) / math.sqrt(D)
                if c["cap"]:
                    sc = c["cap"] * torch.tanh(sc / c["cap"])
                if c["bias"]:
                    sc = sc - s["slopes"][h * G : (h + 1) * G].double()[None, :, None] * (p[t0:t1] - j[None]).abs()[:, None]
                sc = torch.where(see[t0:t1, None], sc, -torch.inf)
                top = sc.amax(-1, keepdim=True)
                w = torch.exp(sc - torch.where(torch.isfinite(top), top, 0.0))
                total = w.sum(-1, keepdim=True)
                r = (w.reshape(-1, length + n) @ V).reshape(t1 - t0, G, D)
                out[first + t0 : first + t1, h * G : (h + 1) * G] = torch.where(total > 0, r / total, 0.0)
        first += n
    return out


def _exact_advance(c, s):
    table, uses, page = s["table"].cpu().numpy().copy(), s["uses"].cpu().numpy().copy(), c["page"]
    free, lacking = list(np.flatnonzero(uses <= 0)), 0
    free.reverse()
    for b, (n, length) in enumerate(zip(_counts(c), _lens(c))):
        end = min(length + n, table.shape[1] * page)
        for i in np.flatnonzero(table[b] >= 0):
            seen = c["window"] == 0 or i * page < c["sinks"] or (i + 1) * page > length - c["window"] + 1
            if i * page >= end or not seen:
                uses[table[b, i]] -= 1
                table[b, i] = -1
        for i in range(-(-length // page), -(-end // page)):
            seen = c["window"] == 0 or i * page < c["sinks"] or (i + 1) * page > length - c["window"] + 1
            if table[b, i] < 0 and seen:
                if free:
                    table[b, i] = free.pop()
                    uses[table[b, i]] = 1
                else:
                    lacking += 1
    return torch.from_numpy(table).cuda(), torch.from_numpy(uses).cuda(), _ints([lacking])


def _moved(s, moves):
    out = []
    for pools in s["pools"]:
        for p in pools:
            q = p.double()
            if moves:
                src, dst = (torch.tensor([m[i] for m in moves], device="cuda") for i in (0, 1))
                q[dst] = p[src].double()
            out.append(q)
    return out


def _exact_fork(c, s):
    table, uses, lens = s["table"].cpu().numpy(), s["uses"].cpu().numpy(), _lens(c)
    out, free, seen = np.full_like(table, -1), list(np.flatnonzero(uses <= 0)), set()
    copies, lens_out, lacking = [[-1, -1] for _ in lens], [0] * len(lens), 0
    for b, p in enumerate(_parents(c)):
        if p < 0:
            continue
        lens_out[b] = lens[p]
        if p not in seen:
            seen.add(p)
            out[b] = table[p]
            continue
        whole = lens[p] // c["page"]
        out[b, :whole] = table[p, :whole]
        if lens[p] % c["page"]:
            if free:
                out[b, whole] = free.pop(0)
                copies[b] = [int(table[p, whole]), int(out[b, whole])]
            else:
                lacking += 1
    named = np.bincount(out[out >= 0], minlength=len(uses)) - np.bincount(table[table >= 0], minlength=len(uses))
    return [torch.from_numpy(out).cuda(), torch.from_numpy((uses + named).astype(np.int32)).cuda(), _ints(copies),
            _ints([lacking]), _ints(lens_out)] + _moved(s, [m for m in copies if m[0] >= 0])


def _exact_compact(c, s):
    table, uses = s["table"].cpu().numpy().copy(), s["uses"].cpu().numpy().copy()
    live = int((uses > 0).sum())
    moves = list(zip(np.flatnonzero(uses[live:] > 0)[::-1] + live, np.flatnonzero(uses[:live] <= 0)))
    to = np.arange(len(uses), dtype=np.int32)
    for a, b in moves:
        to[a], uses[b], uses[a] = b, uses[a], 0
    table[table >= 0] = to[table[table >= 0]]
    copies = [[int(a), int(b)] for a, b in moves] + [[-1, -1]] * (len(uses) // 2 - len(moves))
    return [torch.from_numpy(table).cuda(), torch.from_numpy(uses).cuda(), _ints(copies).view(-1, 2), _ints([live])] + _moved(
        s, [m for m in copies if m[0] >= 0])
