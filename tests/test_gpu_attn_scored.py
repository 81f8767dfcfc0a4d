"""Attention with shaped scores and ranges of rows (bdssm_attn_step_ex) against the definition in
float64 numpy, element by element.

Bounds, from the arithmetic (e = 2^-24). With S the largest scale * sum_d |q_d k_d| of a query: a
float32 score errs by (D + 8) e S as in plain attention; a cap passes that on at most (tanh's
slope is 1 at most) and adds its own rounding, at most 12 e of a result that S bounds; a bias
slope * d (d counted from the nearest visible position, exact) adds 4 e (S + slope d), and the
power's argument, the difference to the maximum, 4 e of its magnitude. So a weight errs by
E_j = e ((D + 40) S + 8 slope d_j) relatively, their sum by the mean of that, sums over n keys by
n e. With bf16 values each weight is rounded (2^-8 at most), and so is the result (half a unit)."""
import numpy as np
import pytest

from bidirectional_mamba_state_amd import bdssm
from test_gpu_attn import BF16, F32, Case, _case, _np, half_ulp

pytestmark = pytest.mark.gpu


def slopes_of(H):
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


def documents(lens, counts, borders):
    """(first, last) of every chunk row: the borders around its position."""
    first, last = [], []
    for L, n in zip(lens, counts):
        for p in range(L, L + n):
            i = int(np.searchsorted(borders, p, side="right"))
            first.append(0 if i == 0 else borders[i - 1])
            last.append(borders[i] if i < len(borders) else 2**31 - 1)
    return first, last


class Scored(Case):
    def __init__(self, lens, counts, cap=0.0, slopes=None, prefix=None, first=None, last=None, **kw):
        import torch
        kw.setdefault("ragged", len(set(counts)) > 1)
        super().__init__(lens, counts, **kw)
        self.cap, self.slopes, self.prefix, self.lo, self.hi = cap, slopes, prefix, first, last
        ints = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        s = None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda")
        self.scores = bdssm.AttnScores(cap, s, ints(prefix), ints(first), ints(last))

    def workspace(self):
        import torch
        need = bdssm.attn_step_ex_workspace(self.ad, self.T, self.max_len, self.mask, self.scores)
        return torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None

    def run(self, stream=None, out=None, ws=None):
        import torch
        fresh = out is None
        if fresh:
            out = torch.full((self.n, self.H, self.D), float("nan"), dtype=self.q.dtype, device="cuda")
            ws = self.workspace()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        bdssm.attn_step_ex(self.ad, self.T, self.q, self.k if self.own_keys else None, self.v if self.own_keys else None,
                           self.cache, self.mask, self.scores, out, ws, starts=self.starts, stream=stream)
        if fresh:
            torch.cuda.synchronize()
        return out

    def want(self):
        G, e = self.H // self.KV, 2.0**-24
        kp, vp, table = _np(self.kp), _np(self.vp), self.table.cpu().numpy()
        q, k, v = _np(self.q), _np(self.k), _np(self.v)
        slopes = None if self.slopes is None else np.float32(self.slopes).astype(np.float64)
        out, tol = np.zeros((self.n, self.H, self.D)), np.zeros((self.n, self.H, self.D))
        for b, (L, n) in enumerate(zip(self.lens, self.counts)):
            r0 = int(self.first[b])
            held = [j for j in range(L) if 0 <= table[b, j // self.page] < kp.shape[0]]
            pos = np.array(held + ([L + i for i in range(n)] if self.own_keys else []), np.int64)
            for h in range(self.KV):
                get = lambda pages, new: np.array([pages[table[b, j // self.page], h, j % self.page] for j in held] +  # noqa: E731
                                                  ([new[r0 + i, h] for i in range(n)] if self.own_keys else [])).reshape(-1, self.D)
                K, V = get(kp, k), get(vp, v)
                for i in range(n):
                    p = L + i
                    see = np.ones(len(pos), bool)
                    if self.block:
                        see &= (pos // self.block <= p // self.block) | (pos < (self.prefix[b] if self.prefix else 0))
                    if self.window:
                        see &= (p - pos < self.window) | (pos < self.sinks)
                    if self.lo is not None:
                        see &= pos >= self.lo[r0 + i]
                    if self.hi is not None:
                        see &= pos < self.hi[r0 + i]
                    if not see.any():
                        continue
                    Ks, Vs, d = K[see], V[see], np.abs(p - pos[see])
                    near = (d - d.min()).astype(np.float64)
                    for gq in range(G):
                        qq = q[r0 + i, h * G + gq]
                        s = self.scale * (Ks @ qq)
                        if self.cap:
                            s = self.cap * np.tanh(s / self.cap)
                        slope = 0.0 if slopes is None else slopes[h * G + gq]
                        s = s - slope * d
                        w = np.exp(s - s.max())
                        w /= w.sum()
                        o, W = w @ Vs, w @ np.abs(Vs)
                        S = self.scale * (np.abs(Ks) @ np.abs(qq)).max()
                        E = e * ((self.D + 40) * S + 8 * abs(slope) * near)
                        t = (w * E) @ np.abs(Vs) + W * ((w @ E) + e * 2 * (len(Ks) + 16))
                        if self.dtype == BF16:
                            t = 1.01 * (t + 2.0**-8 * W)
                            t = t + half_ulp(np.abs(o) + t)
                        out[r0 + i, h * G + gq], tol[r0 + i, h * G + gq] = o, t + 1e-30
        return out, tol


KINDS = {"cap": dict(cap=5.0), "bias": dict(slopes=True), "both": dict(cap=30.0, slopes=True)}


def scored(lens, counts, kind, H=4, **kw):
    more = dict(KINDS[kind])
    if more.get("slopes"):
        more["slopes"] = slopes_of(H)
    return Scored(lens, counts, H=H, **more, **kw)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("lens,counts", [
    ([0], [1]), ([1], [1]), ([300], [1]), ([0], [33]), ([65], [32]), ([200, 0, 17], [32, 32, 32]), ([70], [130])])
def test_lengths(lens, counts, dtype, D, kind):
    _case(f"scored lengths {lens} {counts} dtype {dtype} D {D} {kind}")
    scored(lens, counts, kind, D=D, dtype=dtype).check(kind)


@pytest.mark.parametrize("H,KV", [(1, 1), (8, 1), (5, 1), (40, 8), (33, 1)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_head_layouts(H, KV, dtype):
    _case(f"scored heads {H}/{KV} dtype {dtype}")
    for n in (1, 9, 70):
        scored([90], [n], "both", H=H, KV=KV, dtype=dtype, page=32).check(f"{n} tokens")


@pytest.mark.parametrize("cap", [1e-3, 0.5, 5.0, 50.0, 400.0, 1e5, 1e30])
@pytest.mark.parametrize("qscale", [0.01, 2.0, 30.0])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_caps(cap, qscale, dtype):
    _case(f"cap {cap} qscale {qscale} dtype {dtype}")
    Scored([100], [20], cap=cap, qscale=qscale, dtype=dtype).check("cap")


@pytest.mark.parametrize("cap", [0.5, 8.0, 30.0, 50.0, 256.0, 257.0])
@pytest.mark.parametrize("D", [64, 128])
def test_caps_on_every_bf16_shape(cap, D):
    """Small scores (made along with the weights at headdim 128), large ones and both in one tile, in the
    shapes for few rows, for many, and for many with ranges."""
    _case(f"caps D {D} cap {cap}")
    for qscale in (0.05, 2.0, 8.0):
        Scored([200], [3], H=4, KV=1, D=D, cap=cap, qscale=qscale).check("few rows")
        Scored([130], [150], H=2, KV=1, D=D, cap=cap, qscale=qscale, block=1).check("many rows")
        Scored([130], [90], H=2, KV=1, D=D, cap=cap, qscale=qscale, first=[64] * 90).check("with ranges")
    c = Scored([200], [40], H=4, KV=1, D=D, cap=cap, qscale=0.05)
    c.q[7:20] *= 100  # some rows' scores are large
    c.check("mixed rows")


@pytest.mark.parametrize("slope", [0.0, 1e-4, 0.7, 30.0, -0.01])
@pytest.mark.parametrize("block,window,sinks", [(0, 0, 0), (1, 0, 0), (32, 50, 4)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_slopes(slope, block, window, sinks, dtype):
    _case(f"slope {slope} block {block} window {window} dtype {dtype}")
    Scored([150], [70], slopes=[slope] * 4, block=block, window=window, sinks=sinks, dtype=dtype).check("slope")


def test_many_rows_and_a_split_cache():
    """Every launch shape: many rows of each element type, and one token over ranges that are joined."""
    for dtype, D in ((BF16, 64), (BF16, 128), (F32, 64), (F32, 128)):
        _case(f"large dtype {dtype} D {D}")
        scored([40], [300], "both", H=2, KV=1, D=D, dtype=dtype, block=1).check("many rows")
        c = scored([3000], [1], "both", H=2, KV=1, D=D, dtype=dtype)
        assert c.workspace() is not None
        c.check("split")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("block", [0, 1, 32])
@pytest.mark.parametrize("kind", [None, "both"])
def test_documents(dtype, block, kind):
    """Documents packed into chunks, some shorter than a tile, some across cache and chunk."""
    _case(f"documents block {block} dtype {dtype} {kind}")
    lens, counts = [0, 130, 7], [200, 100, 33]
    first, last = documents(lens, counts, [3, 4, 40, 64, 100, 150, 152, 200, 215])
    more = {} if kind is None else dict(cap=30.0, slopes=slopes_of(4))
    Scored(lens, counts, first=first, last=last, block=block, dtype=dtype, **more).check("documents")
    Scored(lens, counts, first=first, block=block, dtype=dtype, ragged=True, **more).check("first only")
    Scored(lens, counts, last=last, block=block, dtype=dtype, **more).check("last only")


@pytest.mark.parametrize("dtype,D,streams,block", [(BF16, 64, 33, 0), (BF16, 128, 22, 1), (F32, 64, 11, 1)])
def test_sorted_row_tiles(dtype, D, streams, block):
    """More row tiles than the GPU takes at once, sorted by what they walk (tests/scored_plan_check.cc has
    these shapes): documents, padding, streams of none or few tokens."""
    _case(f"sorted dtype {dtype} D {D}")
    lens = [(i * 37) % 90 for i in range(streams)]
    counts = [0 if i == 5 else 3 if i == 6 else 300 - (i * 13) % 200 if i else 300 for i in range(streams)]
    first, last = documents(lens, counts, [3, 4, 40, 64, 100, 150, 152, 200, 215, 300])
    at = 0
    for n in counts:
        for i in range(max(0, n - n // 16), n):
            first[at + i] = last[at + i] = 0
        at += n
    c = Scored(lens, counts, H=8, KV=8, D=D, dtype=dtype, first=first, last=last, block=block, cap=20.0)
    assert c.workspace() is not None
    c.check("sorted")
    assert (c.run() == c.run()).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ranges_over_a_cut_cache(dtype):
    """Few rows on a long cache, their keys cut into ranges of which some hold nothing that they see."""
    _case(f"cut cache dtype {dtype}")
    for first, last in (([0, 2900, 100], [3000, 3003, 101]), ([2000, 2000, 2000], [2010, 2001, 2000])):
        c = Scored([3000], [3], H=2, KV=1, dtype=dtype, first=first, last=last, slopes=[0.5, 0.1])
        assert c.workspace() is not None
        c.check("cut")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 40), (30, 5), (64, 100)])
@pytest.mark.parametrize("own_keys", [True, False])
def test_random_ranges(dtype, window, sinks, own_keys):
    """Any ranges: empty, reversed, past both ends, behind the window, only sinks left."""
    _case(f"random ranges window {window} sinks {sinks} own {own_keys} dtype {dtype}")
    g = np.random.default_rng(window + sinks + own_keys)
    lens, counts = [170, 0, 64], [90, 80, 64]
    n = sum(counts)
    first = g.integers(-20, 260, n)
    last = first + g.integers(-30, 200, n)
    first[::7], last[::7] = 0, 5
    first[3::11], last[3::11] = 0, 0
    first[5::13], last[5::13] = -2**31, 2**31 - 1
    first[6::17], last[6::17] = 2**31 - 1, -2**31
    c = Scored(lens, counts, first=list(map(int, first)), last=list(map(int, last)), window=window, sinks=sinks, block=1,
               slopes=slopes_of(4), own_keys=own_keys, dtype=dtype)
    c.check("ranges")
    out, empty = c.run(), [i for i in range(n) if last[i] <= first[i]]
    assert (out[empty] == 0).all()


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (F32, 64)])
def test_rows_without_a_range_beside_others(dtype, D):
    """Padding at the end of a chunk, a whole chunk of it, and a stream of it between others."""
    _case(f"padding dtype {dtype}")
    lens, counts = [300, 20, 5], [280, 40, 60]
    first, last = [0] * sum(counts), [2**31 - 1] * sum(counts)
    for i in list(range(250, 280)) + list(range(280, 320)):
        last[i] = 0
    Scored(lens, counts, first=first, last=last, D=D, dtype=dtype, cap=20.0, block=1).check("padding")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("block", [0, 1, 32])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_prefix(dtype, block, window, sinks):
    _case(f"prefix block {block} window {window} dtype {dtype}")
    for prefix in ([0, 50, 150, -3], [2**31 - 1, 64, 100, 1]):
        Scored([0, 0, 100, 64], [100, 128, 90, 33], prefix=prefix, block=block, window=window, sinks=sinks,
               dtype=dtype).check(f"prefix {prefix}")
    first, last = documents([30], [120], [10, 50, 90, 140])
    Scored([30], [120], prefix=[100], first=first, last=last, block=block, dtype=dtype).check("with documents")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_infinities_stay_with_their_document(dtype):
    """Values of one document's keys that are infinite or NaN reach its own rows and no others."""
    import torch
    _case(f"infinities dtype {dtype}")
    lens, counts = [100], [150]
    first, last = documents(lens, counts, [60, 120, 121, 200])
    make = lambda: Scored(lens, counts, first=first, last=last, block=0, cap=10.0, slopes=slopes_of(4), dtype=dtype)  # noqa: E731
    plain = make().run()
    for at, bad in ((70, float("inf")), (130 - 100, float("nan")), (220 - 100, float("-inf"))):
        c = make()
        if at == 70:
            c.vp[c.table[0, at // c.page], :, at % c.page] = bad
            p = at
        else:
            c.v[at] = bad
            p = at + 100
        got = c.run()
        sees = torch.tensor([f <= p < l for f, l in zip(first, last)], device="cuda")
        assert not torch.isfinite(got[sees]).any()
        assert torch.isfinite(got[~sees]).all()
        diff = (got[~sees].float() - plain[~sees].float()).abs().max().item()
        # the weights may be rounded from another reference: a unit of bf16 of a value of 4 or so
        assert diff <= (2.0**-5 if dtype == BF16 else 1e-4), diff


def test_infinite_scores_under_a_cap():
    """A cap makes a score finite whose sum of products overflows: 1e30 x 1e30 does, with one sign
    (products that overflow with both signs add up to inf - inf, a NaN, in any order), and 1e30 x
    the other numbers, below 10, does not."""
    _case("infinite scores")
    for dtype in (BF16, F32):
        for sign in (1.0, -1.0):
            c = Scored([40], [8], cap=3.0, dtype=dtype)
            c.q[3] = 1e30
            c.kp[c.table[0, 1], :, 2] = sign * 1e30
            c.check(f"infinite {sign}")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_range_far_from_the_query(dtype):
    """Where every visible key is far away the common distance leaves no trace."""
    _case(f"far range dtype {dtype}")
    L, n = 60000, 5
    c = Scored([L], [n], first=[10] * n, last=[200] * n, slopes=[0.5, 0.3, 0.01, 1.0], dtype=dtype, page=256)
    c.check("far")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_positions_past_2_to_the_24(dtype):
    """A stream of 33 million tokens of which the window's pages are left."""
    import torch
    _case(f"far positions dtype {dtype}")
    L, n, page, window, H, KV, D = (1 << 25) + 77, 6, 256, 300, 2, 1, 64
    td = torch.bfloat16 if dtype == BF16 else torch.float32
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    near = Scored([window + 20], [n], H=H, KV=KV, D=D, dtype=dtype, page=page, block=1, window=window, slopes=[0.4, 0.02])
    # the same keys, all positions moved by L - (window + 20), which is made a multiple of the page
    L = L // page * page + (window + 20) % page + page * 3
    shift = (L - (window + 20)) // page
    assert shift * page + window + 20 == L
    per = -(-(L + n) // page)
    table = torch.full((1, per), -1, dtype=torch.int32, device="cuda")
    table[:, shift:] = near.table[:, :per - shift]
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    cache = bdssm.KvCache(near.ad, near.kp, near.vp, table, lens, L)
    out = torch.empty((n, H, D), dtype=td, device="cuda")
    need = bdssm.attn_step_ex_workspace(near.ad, n, L, near.mask, near.scores)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    bdssm.attn_step_ex(near.ad, n, near.q, near.k, near.v, cache, near.mask, near.scores, out, ws)
    want, tol = near.want()
    assert (np.abs(_np(out) - want) <= tol).all()


def test_without_scores_it_is_attention():
    _case("nothing shaped")
    for dtype in (BF16, F32):
        Scored([100, 30], [40, 40], block=32, window=60, sinks=4, dtype=dtype).check("plain")


def test_rows_past_a_stream_and_other_streams_order():
    """Rows that no stream owns keep what they held; a call on another stream; twice the same bits."""
    import torch
    _case("rows past the last")
    c = scored([50, 20], [30, 10], "both", ragged=True)
    n = c.n + 9
    pad = lambda t: torch.cat([t.contiguous(), torch.full((9, *t.shape[1:]), float("nan"), dtype=t.dtype, device="cuda")])  # noqa: E731
    q, k, v = pad(c.q), pad(c.k), pad(c.v)
    out = torch.full((n, c.H, c.D), 7.0, dtype=q.dtype, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bdssm.attn_step_ex(c.ad, c.T, q, k, v, c.cache, c.mask, c.scores, out, c.workspace(), starts=c.starts, stream=side)
    side.synchronize()
    assert (out[c.n:] == 7.0).all()
    assert torch.equal(out[:c.n], c.run())


def test_graph_replays():
    """Captured and replayed, with eager work in between: the eager result, bit for bit, for the
    cache's changing lengths too."""
    import torch
    _case("graph")
    c = scored([900, 500], [32, 32], "both", H=6, KV=2)
    out = torch.empty((c.n, c.H, c.D), dtype=c.q.dtype, device="cuda")
    ws = c.workspace()
    c.run(out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=out, ws=ws)
    for lens in ([900, 500], [3, 480], [0, 0], [900, 500]):
        c.lens_d.copy_(torch.tensor(lens, dtype=torch.int32))
        want = c.run().clone()
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), lens


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)])
def test_queries_that_a_window_leaves_no_cached_key(dtype, D, kind):
    """Without keys of the chunk's own a window leaves the first queries some of the cache and the later
    ones nothing: zeros, beside rows of the same workgroup that see keys."""
    _case(f"scored cache alone D {D} dtype {dtype} {kind}")
    for lens, counts, more in [([0, 40, 5], [20, 20, 20], {}), ([100], [70], {}), ([100], [70], dict(block=1)),
                               ([3000], [12], {}), ([100], [70], dict(prefix=[30]))]:
        c = scored(lens, counts, kind, dtype=dtype, D=D, own_keys=False, window=10, **more)
        out = c.run()
        c.check("cache alone")
        assert not out[10:20].any()  # row 10 of the first stream looks back to position lens + 1


@pytest.mark.parametrize("own_keys", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_bias_among_sinks_alone(dtype, own_keys):
    """Where the window leaves nothing of the range (or of the cache), distances count from the last
    sink in sight: a steep slope from further back would round the differences away."""
    _case(f"sinks alone dtype {dtype} own keys {own_keys}")
    slopes = [2.0, 0.5, 8.0, 0.0]
    last = [90, 2000, 30, 2**31 - 1, 1999] * 4 if own_keys else None
    for cap in (0.0, 30.0):
        Scored([3000], [20], dtype=dtype, window=9, sinks=40, cap=cap, slopes=slopes, last=last, own_keys=own_keys,
               qscale=0.3).check("sinks alone")
