"""Attention over a paged cache (bdssm_attn_step) and its append (bdssm_kv_append) against the
definition in float64 numpy, element by element.

Bounds, from the arithmetic. With p the exact weights, W = sum_j p_j |v_j| and S the largest
scale * sum_d |q_d k_d| of a query, in float32: a score errs by (D + 8) 2^-24 S at most, its
weight and the weights' sum by twice that relatively, exp by a few 2^-24 (of arguments below
2 S), the sums over n keys by n 2^-24 of W. TOL32 adds these. With bf16 values each weight is
rounded (bf16 has 8 significant bits: 2^-8 relatively at most, so 2^-8 W) and so is the result
(half a unit in its last place)."""
import numpy as np
import pytest

from bidirectional_mamba_state_amd import bdssm

pytestmark = pytest.mark.gpu

F32, BF16 = bdssm.F32, bdssm.BF16


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def half_ulp(v):
    """Half a unit in the last place of a bf16 value of magnitude |v|: 2^(e - 8) in [2^e, 2^(e+1))."""
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0**-126))) - 8)


class Case:
    """Seeded inputs on the device, with NaN in every slot that no query may use: free pages,
    the last page past a stream's length, pages given back under a window."""

    def __init__(self, lens, counts, H=4, KV=2, D=64, dtype=BF16, page=16, block=0, window=0, sinks=0, ragged=False,
                 own_keys=True, drop=(), seed=0, spare=3, qscale=2.0):
        import torch
        self.lens, self.counts, self.H, self.KV, self.D, self.dtype, self.page = lens, counts, H, KV, D, dtype, page
        self.block, self.window, self.sinks, self.own_keys = block, window, sinks, own_keys
        td = torch.bfloat16 if dtype == BF16 else torch.float32
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1000 * sum(lens) + sum(counts))
        b, T = len(lens), max(counts)
        self.b, self.T = b, T
        per = max(1, -(-(max(lens) + T) // page))
        pool = b * per + spare
        shape = (pool, KV, page, D)
        self.kp = torch.full(shape, float("nan"), dtype=td, device="cuda")
        self.vp = torch.full(shape, float("nan"), dtype=td, device="cuda")
        perm = torch.randperm(pool, generator=g, device="cuda")[:b * per].to(torch.int32).reshape(b, per)
        self.table = perm.clone()
        for s, L in enumerate(lens):
            for i in range(-(-L // page)):
                m = min(page, L - i * page)
                self.kp[perm[s, i], :, :m] = torch.randn((KV, m, D), generator=g, device="cuda").to(td)
                self.vp[perm[s, i], :, :m] = torch.randn((KV, m, D), generator=g, device="cuda").to(td)
            for i in range(per):
                lo = max(sinks, 0)
                if window and i * page >= lo and (i + 1) * page <= L - window + 1:
                    self.kp[perm[s, i]] = float("nan")
                    self.vp[perm[s, i]] = float("nan")
                    self.table[s, i] = -1 if i % 2 else pool + 7  # both ways out of range
        for s, i in drop:  # pages that are visible by position, but not held
            self.table[s, i] = -1
        starts = np.concatenate([[0], np.cumsum(counts)])
        self.first = starts
        n = int(starts[-1])
        self.n = n
        qkv = torch.randn((max(n, 1), (H + 2 * KV) * D + 32), generator=g, device="cuda").to(td)[:n]
        self.q = (qkv[:, :H * D] * qscale).to(td).view(n, H, D) if not ragged else qkv[:, :H * D].view(n, H, D)
        self.k = qkv[:, H * D:(H + KV) * D].view(n, KV, D)
        self.v = qkv[:, (H + KV) * D:(H + 2 * KV) * D].view(n, KV, D)
        self.starts = torch.tensor(starts, dtype=torch.int32, device="cuda") if ragged else None
        self.lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.ad = bdssm.attn_dims(b, H, KV, D, dtype, page)
        self.max_len = max(lens)
        self.cache = bdssm.KvCache(self.ad, self.kp, self.vp, self.table, self.lens_d, self.max_len)
        self.scale = D ** -0.5
        self.mask = bdssm.attn_mask(self.scale, block, window, sinks)

    def run(self, stream=None):
        import torch
        out = torch.full((self.n, self.H, self.D), float("nan"), dtype=self.q.dtype, device="cuda")
        need = bdssm.attn_step_workspace(self.ad, self.T, self.max_len, self.mask)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        bdssm.attn_step(self.ad, self.T, self.q, self.k if self.own_keys else None, self.v if self.own_keys else None,
                        self.cache, self.mask, out, ws, starts=self.starts, stream=stream)
        torch.cuda.synchronize()
        return out

    def want(self):
        """(o, bound) of every token and head, float64."""
        G, e = self.H // self.KV, 2.0**-24
        kp, vp, table = _np(self.kp), _np(self.vp), self.table.cpu().numpy()
        q, k, v = _np(self.q), _np(self.k), _np(self.v)
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
                        see &= pos // self.block <= p // self.block
                    if self.window:
                        see &= (p - pos < self.window) | (pos < self.sinks)
                    if not see.any():
                        continue
                    Ks, Vs = K[see], V[see]
                    for gq in range(G):
                        qq = q[r0 + i, h * G + gq]
                        s = self.scale * (Ks @ qq)
                        w = np.exp(s - s.max())
                        w /= w.sum()
                        o, W = w @ Vs, w @ np.abs(Vs)
                        S = self.scale * (np.abs(Ks) @ np.abs(qq)).max()
                        t = W * e * (4 * (self.D + 8) * S + 8 * S + 2 * (len(Ks) + 16))
                        if self.dtype == BF16:
                            t = 1.01 * (t + 2.0**-8 * W)
                            t = t + half_ulp(np.abs(o) + t)
                        out[r0 + i, h * G + gq], tol[r0 + i, h * G + gq] = o, t + 1e-30
        return out, tol

    def check(self, what):
        got = _np(self.run())
        want, tol = self.want()
        assert np.all(np.isfinite(got)), what
        err = np.abs(got - want)
        worst = float(np.max(err / np.maximum(tol, 1e-30))) if got.size else 0.0
        print(f"[parity] {what}: largest error {worst:.3f} of its bound", flush=True)
        assert np.all(err <= np.maximum(tol, 0.0)), what


def _case(msg):
    print(f"[case] {msg}", flush=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,counts", [
    ([0], [1]), ([1], [1]), ([15], [1]), ([16], [1]), ([64], [1]), ([300], [1]), ([0], [33]), ([63], [2]),
    ([65], [32]), ([130], [70]), ([200, 0, 17], [32, 32, 32]), ([70], [130]), ([513], [5])])
def test_lengths(lens, counts, dtype, D):
    _case(f"lengths {lens} {counts} dtype {dtype} D {D}")
    Case(lens, counts, D=D, dtype=dtype).check("lengths")


@pytest.mark.parametrize("H,KV", [(1, 1), (3, 3), (8, 1), (5, 1), (12, 2), (40, 8), (33, 1), (64, 1)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_head_layouts(H, KV, dtype):
    _case(f"heads {H}/{KV} dtype {dtype}")
    Case([90], [9], H=H, KV=KV, dtype=dtype, page=32).check("one stream")
    Case([90], [1], H=H, KV=KV, dtype=dtype, page=32).check("one token")


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pages_ending_inside_a_tile(page, dtype):
    _case(f"page {page}")
    Case([page - 1, page, page + 1, 3 * page + 5, 0], [7] * 5, page=page, dtype=dtype).check("page sizes")


@pytest.mark.parametrize("block", [1, 3, 32, 100])
@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (F32, 64)])
def test_block_order(block, dtype, D):
    _case(f"block {block}")
    Case([0], [150], block=block, dtype=dtype, D=D).check("no prefix")
    Case([77], [150], block=block, dtype=dtype, D=D, H=6, KV=2).check("prefix not a multiple of the block")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (7, 0), (64, 4), (65, 33), (200, 70), (1000, 4), (100000, 3)])
@pytest.mark.parametrize("block", [0, 1, 32])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_windows(window, sinks, block, dtype):
    _case(f"window {window} sinks {sinks} block {block} dtype {dtype}")
    Case([431, 12, 0], [40, 40, 40], block=block, window=window, sinks=sinks, dtype=dtype).check("window")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_window_over_a_long_chunk(dtype):
    _case("window inside the chunk")
    Case([100], [300], block=1, window=37, sinks=5, dtype=dtype, H=2, KV=1).check("causal")
    Case([3], [300], block=1, window=37, sinks=20, dtype=dtype, H=2, KV=1).check("sinks reach into the chunk")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_that_see_nothing(dtype):
    """Without the chunk's keys a query may attend to nothing: an empty cache, a window that the
    later tokens have left, pages that are not held. Its output is zero."""
    import torch
    _case("empty rows")
    c = Case([0, 40, 5], [20, 20, 20], own_keys=False, window=10, dtype=dtype)
    c.check("cache only")
    out = c.run()
    assert torch.count_nonzero(out[:20]) == 0 and torch.count_nonzero(out[30:40]) == 0
    Case([64, 40], [3, 3], own_keys=False, dtype=dtype, drop=[(0, 0), (0, 1), (0, 2), (0, 3), (1, 1)]).check("no pages held")
    Case([300], [3], dtype=dtype, drop=[(0, 0), (0, 5), (0, 18)]).check("some pages not held")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("block,window", [(0, 0), (1, 0), (32, 50)])
def test_ragged_chunks(dtype, block, window):
    _case("ragged")
    Case([50, 0, 333, 128, 7], [5, 0, 64, 1, 33], ragged=True, dtype=dtype, block=block, window=window, sinks=2,
         H=6, KV=2).check("ragged")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts", [[1], [4], [32]])
def test_long_cache(dtype, counts):
    """A cache long enough to be split over workgroups, with one query's scores far above the
    others' in one part only (the join has to weigh parts by their maxima)."""
    _case(f"long cache {counts}")
    c = Case([5000], counts, H=2, KV=1, dtype=dtype, page=64)
    pg = int(c.table[0, 40])
    c.kp[pg, 0, 3] = (c.q[0, 0].float() * 4).to(c.kp.dtype)
    c.check("long")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_scores(dtype):
    """Scores of some hundreds: the running maximum moves, weights vanish or dominate."""
    _case("large scores")
    c = Case([333], [21], dtype=dtype, qscale=30.0)
    c.check("large")


@pytest.mark.parametrize("dtype,D,block", [(BF16, 64, 0), (BF16, 64, 32), (BF16, 128, 1), (F32, 64, 0), (F32, 128, 32)])
def test_many_streams_of_several_row_tiles(dtype, D, block):
    """Streams of 0 to 3 row tiles in one launch, split and not, some without chunk tokens."""
    _case(f"row tiles {dtype} {D} {block}")
    Case([700, 0, 333, 64, 129, 31, 640, 5, 256], [100, 90, 0, 1, 64, 33, 43, 86, 7], H=12, KV=2, D=D, dtype=dtype,
         page=32, block=block, ragged=True).check("row tiles")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("block", [0, 1])
def test_one_kv_head_of_many_rows(dtype, block):
    """One unit with many row tiles: they are dealt to all XCDs."""
    _case(f"many rows {dtype} {block}")
    Case([40], [650], H=4, KV=1, dtype=dtype, block=block).check("many rows")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(0, 0), (900, 4), (2500, 40)])
def test_more_than_64_pages(dtype, window, sinks):
    """Page numbers are kept 64 at a time: caches of more, windows that start past the first 64,
    pages not held among the second 64."""
    _case(f"pages {dtype} {window}")
    Case([3000, 1024, 1040], [20, 20, 20], H=4, KV=2, dtype=dtype, page=16, window=window, sinks=sinks).check("pages")
    Case([3000], [3], H=2, KV=1, dtype=dtype, page=16, window=window, sinks=sinks,
         drop=[(0, i) for i in range(150, 160)]).check("pages not held")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ranges_that_see_nothing(dtype):
    """A long cache split over workgroups where whole ranges hold no page: they join with weight 0,
    and where no range sees anything the result is zero."""
    import torch
    _case("empty ranges")
    Case([5000], [2], H=2, KV=1, dtype=dtype, page=64, own_keys=False, drop=[(0, i) for i in range(0, 50)]).check("some")
    c = Case([5000], [2], H=2, KV=1, dtype=dtype, page=64, own_keys=False, drop=[(0, i) for i in range(0, 79)])
    assert torch.count_nonzero(c.run()) == 0


def test_launch_plans_keep_their_results():
    """The same stream alone (few units: its keys split, its row tiles dealt to all XCDs) and among
    others (many units): the same attention within the bound of each."""
    _case("alone and among others")
    for lens, counts in (([900], [60]), ([900] * 9, [60] * 9)):
        Case(lens, counts, H=16, KV=2, page=32).check(f"{len(lens)} streams")


def test_repeatable_streams_and_extra_rows():
    import torch
    c = Case([1000, 37], [16, 16], H=8, KV=2)
    a, b = c.run(), c.run(torch.cuda.Stream())
    assert torch.equal(a, b)


def test_counts_past_the_bounds_the_host_gave():
    """lens above max_len and below zero, starts past the rows: clamped, nothing out of bounds."""
    import torch
    c = Case([100, 60], [8, 8], ragged=True)
    c.cache.max_len = 64
    c.max_len = 64
    c.lens_d.copy_(torch.tensor([1 << 30, -5], dtype=torch.int32))
    c.starts.copy_(torch.tensor([0, 8, 1 << 30], dtype=torch.int32))
    got = _np(c.run())
    c.lens = [64, 0]
    want, tol = c.want()
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("ragged", [False, True])
def test_append(dtype, D, page, ragged):
    import torch
    _case(f"append {dtype} {D} {page} {ragged}")
    lens, counts = ([0, 5, page, 3 * page - 1], [33, 0, 1, 2 * page + 3]) if ragged else ([0, 5, page], [19, 19, 19])
    c = Case(lens, counts, dtype=dtype, D=D, page=page, ragged=ragged, KV=3, H=3)
    as_int = lambda t: t.view(torch.int16 if dtype == BF16 else torch.int32).clone()  # noqa: E731
    wk, wv = as_int(c.kp), as_int(c.vp)
    for s, (L, n) in enumerate(zip(lens, counts)):
        for i in range(n):
            pg, slot = int(c.table[s, (L + i) // page]), (L + i) % page
            wk[pg, :, slot] = as_int(c.k[int(c.first[s]) + i].contiguous())
            wv[pg, :, slot] = as_int(c.v[int(c.first[s]) + i].contiguous())
    out = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    bdssm.kv_append(c.ad, c.T, c.k, c.v, c.cache, out, starts=c.starts)
    torch.cuda.synchronize()
    assert torch.equal(as_int(c.kp), wk) and torch.equal(as_int(c.vp), wv)
    assert out.tolist() == [L + n for L, n in zip(lens, counts)]
    assert c.lens_d.tolist() == lens


def test_append_past_the_table_and_to_pages_not_held():
    import torch
    c = Case([30, 10], [10, 10], page=16)
    c.table[0, 2] = -1
    c.cache = bdssm.KvCache(c.ad, c.kp, c.vp, c.table[:, :2].contiguous(), c.lens_d, 30)  # two pages each
    before = c.kp.view(torch.int16).clone()
    out = torch.empty(2, dtype=torch.int32, device="cuda")
    bdssm.kv_append(c.ad, 10, c.k, c.v, c.cache, out)
    torch.cuda.synchronize()
    assert out.tolist() == [32, 20]
    changed = (c.kp.view(torch.int16) != before).any(-1).any(1)  # [page, slot]
    p01, p10, p11 = int(c.table[0, 1]), int(c.table[1, 0]), int(c.table[1, 1])
    got = {(int(p), int(s)) for p, s in changed.nonzero()}
    assert got == {(p01, 14), (p01, 15)} | {(p10, s) for s in range(10, 16)} | {(p11, s) for s in range(4)}


def test_append_then_attend():
    """A commit, then a step: the same as attending to the block as a chunk that comes before."""
    import torch
    c = Case([37], [20], H=4, KV=2, block=1)
    whole = c.run()
    lens = torch.empty_like(c.lens_d)
    half = lambda t: t[:8]  # noqa: E731
    bdssm.kv_append(c.ad, 8, half(c.k), half(c.v), c.cache, lens)
    c.cache.set_lens(lens)
    c.cache.max_len = 45
    out = torch.empty_like(whole)[8:]
    need = bdssm.attn_step_workspace(c.ad, 12, 45, c.mask)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    bdssm.attn_step(c.ad, 12, c.q[8:], c.k[8:], c.v[8:], c.cache, c.mask, out, ws)
    torch.cuda.synchronize()
    err = (out.float() - whole[8:].float()).abs().max() / whole[8:].float().abs().max()
    assert err < 2.0**-6  # two roundings to bf16 and the weights' own, apart


def test_offsets_past_32_bits():
    """Pools of more than 2^32 bytes each: pages at their far ends."""
    import torch
    KV, D, page = 8, 128, 256
    per_page = KV * page * D
    pool = (1 << 31) // per_page + 3 + (1 << 30) // per_page  # element offsets past 2^31, bytes past 2^32
    ad = bdssm.attn_dims(1, KV, KV, D, BF16, page)
    kp = torch.zeros((pool, KV, page, D), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros((pool, KV, page, D), dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[pool - 1, 0, pool - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    k = torch.randn((300, KV, D), generator=g, device="cuda").bfloat16()
    v = torch.randn((300, KV, D), generator=g, device="cuda").bfloat16()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = bdssm.KvCache(ad, kp, vp, table, zero, 0)
    bdssm.kv_append(ad, 300, k, v, cache)
    assert torch.equal(kp[pool - 1, :, :], k[:256].transpose(0, 1)) and torch.equal(vp[0, :, :44], v[256:].transpose(0, 1))
    q = torch.randn((4, KV, D), generator=g, device="cuda").bfloat16()
    cache = bdssm.KvCache(ad, kp, vp, table, lens, 300)
    mask = bdssm.attn_mask(D ** -0.5)
    out = torch.empty_like(q)
    need = bdssm.attn_step_workspace(ad, 4, 300, mask)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    bdssm.attn_step(ad, 4, q, None, None, cache, mask, out, ws)
    torch.cuda.synchronize()
    s = np.einsum("thd,jhd->htj", _np(q), _np(k)) * D ** -0.5
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    want = np.einsum("htj,jhd->thd", w, _np(v))
    tol = 1.05 * 2.0**-8 * (np.einsum("htj,jhd->thd", w, np.abs(_np(v))) + np.abs(want))
    assert np.all(np.abs(_np(out) - want) <= tol)
    del kp, vp
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("lens,counts,heads,block,window,sinks", [
    ([100], [96], (2, 2), 32, 0, 0),               # ordered, in the chunk's own tiles
    ([200, 37], [160, 160], (4, 1), 16, 0, 0),     # several row tiles, in the chunk and in a page
    ([300], [70], (2, 1), 0, 48, 0),               # a window that moves on from row to row
    ([300], [260], (2, 2), 8, 100, 5),             # ordered, with a window and sinks
    ([1500, 9], [40, 40], (8, 1), 1, 900, 2),      # split over workgroups
    ([500], [20], (2, 1), 8, 0, 0),                # wavefronts that share rows
    ([500, 3], [10, 12], (2, 1), 4, 0, 0),
])
def test_infinities_and_nan_stay_with_the_rows_that_attend_to_them(dtype, D, lens, counts, heads, block, window, sinks):
    H, KV = heads
    c = Case(lens, counts, H=H, KV=KV, D=D, dtype=dtype, block=block, window=window, sinks=sinks, ragged=True)
    inf, nan = float("inf"), float("nan")
    _case(f"infinities {dtype} {D} {lens} {counts} {block} {window}")
    n = int(c.first[1])
    if block:
        c.v[n - 1, :, 3] = inf
        c.v[n - 1, :, D - 1] = nan
        c.v[n // 2, :, 3] = -inf
        c.v[n // 2, :, 8] = inf
        c.k[n - 2, :, 5] = nan
    if window:
        j = min(lens[0] - window + n // 2, lens[0] - 1)  # some of the rows see it
        pg = int(c.table[0, j // c.page])
        assert pg >= 0
        c.vp[pg, :, j % c.page, 17] = nan
        c.vp[pg, :, j % c.page, 20] = -inf
    got = _np(c.run())
    with np.errstate(invalid="ignore"):
        want, tol = c.want()
    assert (np.isnan(want).any() or np.isinf(want).any()) and np.isfinite(want).all(axis=(1, 2)).any()
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    np.testing.assert_array_equal(np.where(np.isinf(got), got, 0), np.where(np.isinf(want), want, 0))
    ok = np.isfinite(want)
    assert (np.abs(got[ok] - want[ok]) <= tol[ok]).all()
