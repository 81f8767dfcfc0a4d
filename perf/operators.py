"""The attention layer and the norms around the layers of a block-diffusion Mamba hybrid, as
cases to be timed: paged-cache attention of a chunk of new tokens (whole, or through a sliding
window with sinks), the append of a finished chunk to the pages, the gated norm after a scan,
and the residual update with the norms before and after a block.

`listed()` names the cases, `draw()` gives others of the same ranges, `prepare()` makes a case's
inputs on the GPU, `run()` makes one pass (the plain form in elementary torch operations, or
the library's call where `own` is set), `work()` counts the bytes and operations that a pass
cannot do without, `exact()` is the operator's definition in 64 bits.

Head counts and lengths are those of the workload shapes in configs.py (a layer of H heads x 64
belongs to a model of width 32 H: 24, 16 and 40 attention heads of 64 for the 700M, 350M and 3B
shapes; blocks of 32 tokens, running sets of 128, prefixes of 8K to 256K) or generic ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------------------------- cases
def _attn(name, **kw):
    c = dict(name=name, op="attn", batch=1, tokens=32, prefix=8192, heads=24, kv_heads=4, headdim=64, dtype="bf16",
             page=32, ragged=False, block=0, window=0, sinks=0)
    c.update(kw)
    return c


def _append(name, **kw):
    c = dict(name=name, op="append", batch=1, tokens=32, prefix=8192, kv_heads=4, headdim=64, dtype="bf16", page=32,
             ragged=False)
    c.update(kw)
    return c


def _gated(name, **kw):
    c = dict(name=name, op="gated", rows=32, width=2048, groups=1, ydtype="f32", dtype="bf16", norm_first=False)
    c.update(kw)
    return c


def _residual(name, **kw):
    c = dict(name=name, op="residual", batch=1, tokens=32, width=1024, xdtype="f32", dtype="bf16", layer=False,
             post=True, modulate=True)
    c.update(kw)
    return c


def listed():
    return [
        # one token on a short context: a call that is all latency
        _attn("attn_token", tokens=1, prefix=255),
        # a denoising step of the 3B shape's block of 32 over its whole context (5 heads a group)
        _attn("attn_block_long", prefix=262144, heads=40, kv_heads=8),
        # a denoising step of 64 streams, running sets of 4 x 32, prefixes of unequal lengths
        _attn("attn_running_set", batch=64, tokens=128, prefix=32768, page=64, ragged=True),
        # a prompt's second chunk: causal by blocks of 32, heads of 128
        _attn("attn_prompt_chunk", tokens=8192, prefix=8192, heads=20, headdim=128, page=128, block=32),
        # blocks of 64 streams that see 4 first tokens and the last 4096
        _attn("window_block", batch=64, prefix=32768, heads=16, kv_heads=2, ragged=True, window=4096, sinks=4),
        # a prompt in float32, causal, window of 512, one KV head per head, short pages
        _attn("window_prompt_f32", batch=2, tokens=1031, prefix=1000, heads=16, kv_heads=16, dtype="f32", page=16,
              block=1, window=512, sinks=4, ragged=True),
        # the commit of one stream's block, and of long prompts of unequal lengths
        _append("append_block", heads=40, kv_heads=8),
        _append("append_prompts", batch=4, tokens=16384, prefix=1000, kv_heads=8, headdim=128, page=64, ragged=True),
        # after the scan: one block, and the 65,536-token prompt of the 350M shape
        _gated("gated_block"),
        _gated("gated_prompt", rows=65536, ydtype="bf16", groups=8),
        # around a layer: one block's step under a timestep, and a long prompt, plain
        _residual("residual_block", width=2560),
        _residual("residual_prompt", batch=2, tokens=32768, xdtype="bf16", post=False, modulate=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "window", "append", "gated", "residual"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    ragged = rng.random() < 0.5
    if op in ("attn", "window"):
        kv = rng.choice([1, 2, 4, 8])
        c = dict(op="attn", batch=_log(rng, 1, 64), tokens=_log(rng, 1, 4096), prefix=_log(rng, 1, 65536),
                 heads=kv * rng.choice([1, 2, 3, 4, 5, 8]), kv_heads=kv, headdim=rng.choice([64, 128]), dtype=dtype,
                 page=rng.choice([16, 32, 64, 128, 256]), ragged=ragged, block=rng.choice([0, 1, 32]),
                 window=_log(rng, 1, 8192) if op == "window" else 0, sinks=rng.choice([0, 1, 4, 33]) if op == "window" else 0)
        # no costlier than the largest listed cases: their products (float32 has a sixteenth of
        # the matrix rate) and their pages
        while c["batch"] * c["heads"] * c["tokens"] * (c["prefix"] + c["tokens"]) > (1.9e9 if dtype == "bf16" else 2e8):
            c["tokens" if c["tokens"] > 128 else "prefix" if c["prefix"] > 4096 else "batch" if c["batch"] > 1 else "prefix"] //= 2
        while c["batch"] * kv * (c["prefix"] + c["tokens"]) * c["headdim"] > 2.5e8:
            c["prefix"] //= 2
        return c
    if op == "append":
        c = dict(op="append", batch=_log(rng, 1, 64), tokens=_log(rng, 1, 16384), prefix=_log(rng, 1, 16384),
                 kv_heads=rng.choice([1, 2, 4, 8]), headdim=rng.choice([64, 128]), dtype=dtype,
                 page=rng.choice([16, 32, 64, 128, 256]), ragged=ragged)
        while c["batch"] * c["kv_heads"] * (c["prefix"] + c["tokens"]) * c["headdim"] > 6e7:
            c["batch"] = max(1, c["batch"] // 2)
            c["tokens"] = max(1, c["tokens"] // 2)
        return c
    width = _log(rng, 64, 8192)
    rows = min(_log(rng, 1, 65536), 134217728 // width)
    if op == "gated":
        groups = rng.choice([1, 1, 2, 8])
        return dict(op="gated", rows=rows, width=max(groups, width // groups * groups), groups=groups,
                    ydtype=rng.choice(["f32", dtype]), dtype=dtype, norm_first=rng.random() < 0.3)
    batch = rng.choice([1, 2, 5, 64])
    return dict(op="residual", batch=batch, tokens=max(1, rows // batch), width=width, xdtype=rng.choice(["f32", dtype]),
                dtype=dtype, layer=rng.random() < 0.4, post=rng.random() < 0.5, modulate=rng.random() < 0.5)


# ------------------------------------------------------------------- lengths (from the case)
def _counts(c):
    """New tokens of each stream: `tokens`, or where ragged down to half of it (one of several
    streams has none)."""
    T, n = c["tokens"], c["batch"]
    if not c["ragged"]:
        return [T] * n
    return [0 if i == 1 and n > 2 else T - (i * 7919 + 13) % (T // 2 + 1) for i in range(n)]


def _lens(c):
    """Cached tokens of each stream: `prefix`, or where ragged down to half of it."""
    L, n = c["prefix"], c["batch"]
    if not c["ragged"]:
        return [L] * n
    return [L - (i * 6271) % (L // 2 + 1) for i in range(n)]


def _visible(c, n, length):
    """(query, key) pairs that the mask leaves of a stream with n new tokens after `length`
    cached ones, and how many different keys they touch."""
    if n == 0:
        return 0, 0
    blk, win, sinks, end = c["block"], c["window"], c["sinks"], length + n
    pairs, lo_min, hi_max = 0, end, 0
    for p in range(length, end):
        hi = min(end, (p // blk + 1) * blk) if blk else end
        lo = max(0, p - win + 1) if win else 0
        pairs += hi - lo + min(sinks, lo)
        lo_min, hi_max = min(lo_min, lo), max(hi_max, hi)
    return pairs, hi_max - lo_min + min(sinks, lo_min)


def work(c):
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "attn":
        pairs = keys = 0
        for n, length in zip(_counts(c), _lens(c)):
            p, k = _visible(c, n, length)
            pairs, keys = pairs + p, keys + k
        io = 2 * sum(_counts(c)) * c["heads"] * c["headdim"] * e  # queries and outputs
        return {"bytes": io + 2 * keys * c["kv_heads"] * c["headdim"] * e,
                "flops": 4 * pairs * c["heads"] * c["headdim"]}
    if c["op"] == "append":
        return {"bytes": 4 * sum(_counts(c)) * c["kv_heads"] * c["headdim"] * e, "flops": 0}
    if c["op"] == "gated":
        n, ye = c["rows"] * c["width"], 2 if c["ydtype"] == "bf16" else 4
        return {"bytes": n * (ye + 2 * e) + 4 * c["width"], "flops": 10 * n}
    n, xe = c["batch"] * c["tokens"] * c["width"], 2 if c["xdtype"] == "bf16" else 4
    params = 4 * c["width"] * (1 + c["post"]) + 3 * c["batch"] * c["width"] * e * c["modulate"]
    return {"bytes": n * (2 * xe + 2 * e) + params, "flops": 12 * n}


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _cache(c, g):
    """A pool of pages in random order with each stream's table. Under a window the pages that
    no query will see again have been given back: their entries are -1."""
    dt, page, D = DTYPES[c["dtype"]], c["page"], c["headdim"]
    counts, lens = _counts(c), _lens(c)
    per = -(-(c["prefix"] + c["tokens"]) // page)
    pool = c["batch"] * per + 3
    shape = (pool, c["kv_heads"], page, D)
    k, v = _randn(g, shape, dt), _randn(g, shape, dt)
    table = torch.randperm(pool, generator=g, device="cuda")[: c["batch"] * per].to(torch.int32).reshape(c["batch"], per)
    lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if c.get("window"):
        first = torch.arange(per, device="cuda") * page
        gone = (first[None] >= c["sinks"]) & (first[None] + page <= lens_d[:, None] - c["window"] + 1)
        table = torch.where(gone, torch.full_like(table, -1), table)
    starts = None
    if c["ragged"]:
        starts = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    return k, v, table, lens_d, starts, sum(counts)


def prepare(c, seed):
    g = _gen(seed)
    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] in ("attn", "append"):
        D, kv, H = c["headdim"], c["kv_heads"], c["heads"] if c["op"] == "attn" else 0
        kp, vp, table, lens, starts, n = _cache(c, g)
        # queries, keys and values are slices of one projection's rows
        qkv = _randn(g, (n, (H + 2 * kv) * D), dt)
        qkv[:, : H * D] *= 2.0
        s.update(k_pages=kp, v_pages=vp, table=table, lens=lens, starts=starts, n=n,
                 q=qkv[:, : H * D].view(n, H, D) if H else None,
                 k=qkv[:, H * D : (H + kv) * D].view(n, kv, D), v=qkv[:, (H + kv) * D :].view(n, kv, D),
                 out=torch.empty((n, H, D), dtype=dt, device="cuda") if H else None,
                 lens_out=torch.empty_like(lens))
    elif c["op"] == "gated":
        n, w = c["rows"], c["width"]
        zx = _randn(g, (n, 2 * w), dt)  # the gate is one slice of the input projection's rows
        s.update(y=_randn(g, (n, w), DTYPES[c["ydtype"]]), z=zx[:, w:], weight=1 + 0.1 * _randn(g, (w,), torch.float32),
                 out=torch.empty((n, w), dtype=dt, device="cuda"))
    else:
        n, w, b = c["batch"] * c["tokens"], c["width"], c["batch"]
        mod = _randn(g, (b, 3 * w), dt, 0.5) if c["modulate"] else None
        part = lambda i: None if mod is None else mod[:, i * w : (i + 1) * w]  # noqa: E731
        s.update(x=_randn(g, (n, w), DTYPES[c["xdtype"]], 2.0), o=_randn(g, (n, w), dt),
                 post_w=1 + 0.1 * _randn(g, (w,), torch.float32) if c["post"] else None,
                 pre_w=1 + 0.1 * _randn(g, (w,), torch.float32), gate=part(0), gain=part(1), shift=part(2),
                 x_out=torch.empty((n, w), dtype=DTYPES[c["xdtype"]], device="cuda"),
                 u=torch.empty((n, w), dtype=dt, device="cuda"))
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a program of the library keeps beside its tensors: descriptors and a workspace."""
    from bidirectional_mamba_state_amd import bdssm
    c = s["case"]
    dt = bdssm.BF16 if c["dtype"] == "bf16" else bdssm.F32
    if c["op"] in ("attn", "append"):
        s["dims"] = bdssm.attn_dims(c["batch"], c.get("heads", c["kv_heads"]), c["kv_heads"], c["headdim"], dt, c["page"])
        s["cache"] = bdssm.KvCache(s["dims"], s["k_pages"], s["v_pages"], s["table"], s["lens"], c["prefix"])
        if c["op"] == "attn":
            s["mask"] = bdssm.attn_mask(c["headdim"] ** -0.5, c["block"], c["window"], c["sinks"])
            need = bdssm.attn_step_workspace(s["dims"], c["tokens"], c["prefix"], s["mask"])
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    elif c["op"] == "gated":
        s["dims"] = bdssm.norm_dims(c["rows"], c["width"], dt, groups=c["groups"], eps=EPS,
                                    x_dtype=bdssm.BF16 if c["ydtype"] == "bf16" else bdssm.F32)
    else:
        s["dims"] = bdssm.norm_dims(c["batch"] * c["tokens"], c["width"], dt, eps=EPS, rows_per_stream=c["tokens"],
                                    kind=bdssm.NORM_LAYER if c["layer"] else bdssm.NORM_RMS,
                                    x_dtype=bdssm.BF16 if c["xdtype"] == "bf16" else bdssm.F32)


# -------------------------------------------------------------------------------------- runs
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    from bidirectional_mamba_state_amd import bdssm
    c = s["case"]
    if c["op"] == "attn":
        bdssm.attn_step(s["dims"], c["tokens"], s["q"], s["k"], s["v"], s["cache"], s["mask"], s["out"], s["ws"],
                        starts=s["starts"])
        return s["out"]
    if c["op"] == "append":
        bdssm.kv_append(s["dims"], c["tokens"], s["k"], s["v"], s["cache"], s["lens_out"], starts=s["starts"])
        return s["k_pages"], s["v_pages"], s["lens_out"]
    if c["op"] == "gated":
        bdssm.gated_norm(s["dims"], s["y"], s["z"], s["weight"], s["out"], norm_first=c["norm_first"])
        return s["out"]
    bdssm.residual_norm(s["dims"], s["x"], s["o"], s["pre_w"], s["x_out"], s["u"], post_w=s["post_w"], gate=s["gate"],
                        gain=s["gain"], shift=s["shift"], res_scale=0.5)
    return s["x_out"], s["u"]


def _run_plain(s):
    return {"attn": _plain_attn, "append": _plain_append, "gated": _plain_gated, "residual": _plain_residual}[s["case"]["op"]](s)


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
        see = see & (pos[:, None] // c["block"] <= qpos[:, :, None] // c["block"])
    if c["window"]:
        see = see & ((qpos[:, :, None] - pos[:, None] < c["window"]) | (pos[:, None] < c["sinks"]))
    q = s["q"][rows].float().view(b, T, kv, G, D).permute(0, 2, 3, 1, 4).reshape(b, kv, G * T, D)
    p = torch.matmul(q * D ** -0.5, keys(s["k_pages"], s["k"]).transpose(2, 3).contiguous()).view(b, kv, G, T, L + T)
    p.masked_fill_(~see[:, None, None], float("-inf"))
    p.sub_(p.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, kv, G * T, L + T), keys(s["v_pages"], s["v"]).masked_fill_(~ok[:, None, :, None], 0.0))
    o = o.view(b, kv, G, T, D) / total.masked_fill_(total == 0, 1.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(b * T, H, D).to(s["q"].dtype)
    if s["starts"] is None:
        return o
    # back to the tokens' own order: stream of a token, and its place there
    tok = torch.arange(s["n"], device=dev)
    of = torch.searchsorted(st[1:].contiguous(), tok, right=True)
    return o[of * T + tok - st[of]]


def _plain_append(s):
    c = s["case"]
    tok = torch.arange(s["n"], device=s["k"].device)
    if s["starts"] is None:
        of, st = tok // c["tokens"], torch.arange(c["batch"] + 1, device=tok.device) * c["tokens"]
    else:
        st = s["starts"].long()
        of = torch.searchsorted(st[1:].contiguous(), tok, right=True)
    pos = s["lens"].long()[of] + tok - st[of]
    page, slot = s["table"].long()[of, pos // c["page"]], pos % c["page"]
    s["k_pages"][page, :, slot] = s["k"]
    s["v_pages"][page, :, slot] = s["v"]
    torch.add(s["lens"], (st[1:] - st[:-1]).to(torch.int32), out=s["lens_out"])
    return s["k_pages"], s["v_pages"], s["lens_out"]


def _normed(v, layer=False):
    if layer:
        v = v - v.mean(-1, keepdim=True)
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def _plain_gated(s):
    c = s["case"]
    y, z = s["y"].float(), s["z"].float()
    gate = z / (1 + torch.exp(-z))
    part = lambda v: v.view(c["rows"], c["groups"], -1)  # noqa: E731
    if c["norm_first"]:
        r = _normed(part(y)).view_as(y) * s["weight"] * gate
    else:
        r = _normed(part(y * gate)).view_as(y) * s["weight"]
    return r.to(s["out"].dtype)


def _plain_residual(s):
    c = s["case"]
    by = lambda m: m.float().repeat_interleave(c["tokens"], dim=0)  # noqa: E731
    t = s["o"].float()
    if c["post"]:
        t = _normed(t, c["layer"]) * s["post_w"]
    if c["modulate"]:
        t = t * by(s["gate"])
    r = s["x"].float() + 0.5 * t
    u = _normed(r, c["layer"]) * s["pre_w"]
    if c["modulate"]:
        u = u * by(s["gain"]) + by(s["shift"])
    return r.to(s["x"].dtype), u.to(s["o"].dtype)


# ------------------------------------------------------------------------------------- exact
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(c, s)
    if c["op"] == "attn":
        return _exact_attn(c, s)
    if c["op"] == "gated":
        y, z, w = s["y"].double(), s["z"].double(), s["weight"].double()
        shape = (c["rows"], c["groups"], c["width"] // c["groups"])
        g = z * torch.sigmoid(z)
        v = y if c["norm_first"] else y * g
        rms = ((v.reshape(shape) ** 2).sum(-1, keepdim=True) / shape[2] + EPS) ** 0.5
        v = (v.reshape(shape) / rms).reshape(y.shape) * w
        return v * g if c["norm_first"] else v
    n, w, T = c["batch"] * c["tokens"], c["width"], c["tokens"]

    def norm(v):
        mu = v.sum(-1, keepdim=True) / w if c["layer"] else 0.0
        return (v - mu) / (((v - mu) ** 2).sum(-1, keepdim=True) / w + EPS) ** 0.5

    t = s["o"].double().reshape(c["batch"], T, w)
    if c["post"]:
        t = norm(t) * s["post_w"].double()
    if c["modulate"]:
        t = t * s["gate"].double()[:, None]
    r = s["x"].double().reshape(c["batch"], T, w) + 0.5 * t
    u = norm(r) * s["pre_w"].double()
    if c["modulate"]:
        u = u * s["gain"].double()[:, None] + s["shift"].double()[:, None]
    return r.reshape(n, w), u.reshape(n, w)


def _exact_append(c, s):
    k, v = s["k_pages"].clone(), s["v_pages"].clone()
    table, first, lens = s["table"].tolist(), 0, _lens(c)
    for b, n in enumerate(_counts(c)):
        t = 0
        while t < n:  # a page's worth of tokens at a time
            page, slot = divmod(lens[b] + t, c["page"])
            m = min(n - t, c["page"] - slot)
            for pages, new in ((k, s["k"]), (v, s["v"])):
                pages[table[b][page], :, slot : slot + m] = new[first + t : first + t + m].transpose(0, 1)
            t += m
        first += n
    lens_out = torch.tensor([a + b for a, b in zip(lens, _counts(c))], dtype=torch.int32, device="cuda")
    return k.double(), v.double(), lens_out


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
            see = see & (j[None] < (p // c["block"] + 1) * c["block"])
        if c["window"]:
            see = see & ((j[None] > p - c["window"]) | (j[None] < c["sinks"]))
        for h in range(kv if n else 0):
            K, V = (torch.cat([pages[ids.clamp(min=0), h].reshape(-1, D)[:length].double(),
                               new[first : first + n, h].double()]) for pages, new in ((s["k_pages"], s["k"]), (s["v_pages"], s["v"])))
            for t0 in range(0, n, 1024):
                t1 = min(n, t0 + 1024)
                q = s["q"][first + t0 : first + t1, h * G : (h + 1) * G].double()
                sc = (q.reshape(-1, D) @ K.t()).reshape(t1 - t0, G, -1) / math.sqrt(D)
                sc = torch.where(see[t0:t1, None], sc, -torch.inf)
                out[first + t0 : first + t1, h * G : (h + 1) * G] = (torch.softmax(sc, -1).reshape(-1, length + n) @ V).reshape(t1 - t0, G, D)
        first += n
    return out
