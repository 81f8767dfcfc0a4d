"""Rotary positions (bdssm_rotary_step, bdssm_rotary_append) against the definition with angles in
80-bit and products in 64-bit floats, element by element.

Bounds (e = 2^-24): the angle left after whole quarter turns is at most pi / 4 and is rounded three
times (2.4 e), its sine and cosine add 2 e, the scale e, product and sum 2 e of |a| + |b|: 8 e
scale (|a| + |b|). A position's angle is off by 2 pi |p| 2^-65, below e / 100 for positions of 31
bits. With bf16 the result is rounded once more: half a unit in its last place."""
import numpy as np
import pytest

from bidirectional_mamba_state_amd import bdssm
from test_gpu_attn import BF16, F32, _case, _np, half_ulp

pytestmark = pytest.mark.gpu

KINDS = dict(plain=dict(), linear=dict(kind=bdssm.ROTARY_LINEAR, factor=4.0),
             base=dict(kind=bdssm.ROTARY_BASE, factor=8.0),
             parts=dict(kind=bdssm.ROTARY_PARTS, factor=32.0, trained=8192, low=1.0, high=4.0))


def frequencies(dim, base=10000.0, kind=bdssm.ROTARY_PLAIN, factor=1.0, trained=0, low=1.0, high=32.0):
    ld = np.longdouble
    base, s = ld(base), ld(factor)
    if kind == bdssm.ROTARY_BASE:
        base = base * s ** (ld(dim) / ld(dim - 2))
    f = base ** (-2 * np.arange(dim // 2, dtype=ld) / ld(dim))
    if kind == bdssm.ROTARY_LINEAR:
        f = f / s
    if kind == bdssm.ROTARY_PARTS:
        g = np.clip((trained * f / (2 * np.pi) - low) / (high - low), 0, 1)
        f = f * (g + (1 - g) / s)
    return f


def turned(x, pos, f, interleaved, scale):
    """(result, bound without the last rounding) of x [n, heads, D], float64."""
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    t = np.mod(np.asarray(pos).astype(np.longdouble)[:, None] * f[None], two_pi).astype(np.float64)[:, None]
    h = len(f)
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
    y, tol = x.copy(), np.zeros_like(x)
    y[..., a] = scale * (x[..., a] * np.cos(t) - x[..., b] * np.sin(t))
    y[..., b] = scale * (x[..., a] * np.sin(t) + x[..., b] * np.cos(t))
    tol[..., a] = tol[..., b] = 8 * 2.0**-24 * abs(scale) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, tol


def near(got, want, tol, dtype, what):
    got = _np(got)
    if dtype == BF16:
        tol = np.where(tol > 0, tol + half_ulp(np.abs(want) + tol), 0)
    err = np.abs(got - want)
    assert np.all(err <= tol), (what, float(np.max(err - tol)))


class Rows:
    def __init__(self, lens, counts, H=4, KV=2, D=64, dtype=BF16, page=16, seed=0, ragged=True, spare=2, extra=16):
        import torch
        self.lens, self.counts, self.H, self.KV, self.D, self.dtype, self.page = lens, counts, H, KV, D, dtype, page
        self.td = torch.bfloat16 if dtype == BF16 else torch.float32
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 7 * sum(counts) + sum(lens))
        n = self.n = sum(counts)
        self.T = max(counts)
        self.qkv = torch.randn((n, (H + 2 * KV) * D + extra), generator=g, device="cuda").to(self.td)
        self.q, self.k, self.v = self.slices(self.qkv)
        st = np.concatenate([[0], np.cumsum(counts)])
        self.starts = torch.tensor(st, dtype=torch.int32, device="cuda") if ragged else None
        self.lens_d = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.ad = bdssm.attn_dims(len(lens), H, KV, D, dtype, page)
        self.pos = np.concatenate([np.arange(L, L + m) for L, m in zip(lens, counts)]).astype(np.int64)
        per = max(1, -(-max(L + m for L, m in zip(lens, counts)) // page)) if max(lens) < 1 << 20 else 1
        pool = len(lens) * per + spare
        self.table = torch.randperm(pool, generator=g, device="cuda")[:len(lens) * per].to(torch.int32).view(len(lens), per)
        self.kp = torch.full((pool, KV, page, D), 3.0, dtype=self.td, device="cuda")
        self.vp = torch.full((pool, KV, page, D), 4.0, dtype=self.td, device="cuda")

    def slices(self, qkv):
        H, KV, D, n = self.H, self.KV, self.D, self.n
        return (qkv[:, :H * D].view(n, H, D), qkv[:, H * D:(H + KV) * D].view(n, KV, D),
                qkv[:, (H + KV) * D:(H + 2 * KV) * D].view(n, KV, D))

    def cache(self):
        return bdssm.KvCache(self.ad, self.kp, self.vp, self.table, self.lens_d, max(self.lens))

    def check_step(self, dim, interleaved, what, scale=1.0, positions=None, lens="own", **kw):
        import torch
        rot = bdssm.Rotary(bdssm.rotary_turns(dim, **kw), interleaved, scale, positions)
        qo, ko = (torch.full((self.n, h, self.D), float("nan"), dtype=self.td, device="cuda") for h in (self.H, self.KV))
        bdssm.rotary_step(self.ad, self.T, rot, self.q, self.k, qo, ko, lens=self.lens_d if lens == "own" else lens,
                          starts=self.starts)
        f = frequencies(dim, **kw)
        pos = self.pos if positions is None else positions.cpu().numpy().astype(np.int64)
        for got, x in ((qo, self.q), (ko, self.k)):
            near(got, *turned(_np(x), pos, f, interleaved, scale), self.dtype, what)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,dim", [(64, 64), (64, 2), (64, 6), (64, 32), (64, 48), (64, 50), (128, 128), (128, 96), (128, 126),
                                   (128, 8), (128, 16)])
def test_dims(D, dim, interleaved, dtype):
    _case(f"rotary D {D} dim {dim} interleaved {interleaved} dtype {dtype}")
    Rows([0, 300, 17], [1, 20, 7], D=D, dtype=dtype).check_step(dim, interleaved, "dims")


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("interleaved", [False, True])
def test_frequencies(kind, interleaved):
    _case(f"rotary {kind}")
    for dtype in (BF16, F32):
        Rows([131000], [40], dtype=dtype, D=128).check_step(96, interleaved, kind, scale=1.347, **KINDS[kind])


@pytest.mark.parametrize("H,KV,D", [(1, 1, 64), (3, 3, 64), (40, 8, 64), (33, 1, 128), (512, 512, 64)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_heads(H, KV, D, dtype):
    _case(f"rotary heads {H}/{KV} {D}")
    for interleaved in (False, True):
        Rows([5], [3], H=H, KV=KV, D=D, dtype=dtype).check_step(D, interleaved, "heads")


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(interleaved):
    import torch
    _case("rotary far positions")
    r = Rows([0], [300], dtype=F32)
    g = np.random.default_rng(3)
    p = g.integers(-2**31, 2**31, 300)
    p[:6] = [0, -1, 2**31 - 1, -2**31, 2**24 + 1, 262143]
    pos = torch.tensor(p.astype(np.int32), device="cuda")
    for kw in KINDS.values():
        r.check_step(64, interleaved, "far", positions=pos, lens=None, **kw)
    Rows([2**31 - 2000, 1 << 30], [30, 40], dtype=F32).check_step(64, interleaved, "far lengths")
    Rows([0, 0], [30, 40], dtype=F32).check_step(64, interleaved, "no lengths", lens=None)


def test_many_tokens():
    """Workgroups of several tokens, streams that end inside one, even streams without starts."""
    _case("rotary many tokens")
    for dtype in (BF16, F32):
        Rows([3, 900, 5, 0], [7001, 1, 4500, 333], dtype=dtype).check_step(64, False, "ragged")
        Rows([3, 900], [9001, 9001], dtype=dtype, ragged=False).check_step(40, True, "even")
        Rows([0], [40000], H=1, KV=1, dtype=dtype, ragged=False).check_step(36, False, "single pairs")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 20])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_on_slices(dtype, dim, interleaved):
    """In place on slices of one projection: what lies between and behind is left alone."""
    import torch
    _case(f"rotary in place dim {dim}")
    r = Rows([9, 2], [50, 4], dtype=dtype)
    rot = bdssm.Rotary(bdssm.rotary_turns(dim), interleaved)
    qo, ko = torch.empty_like(r.q), torch.empty_like(r.k)
    bdssm.rotary_step(r.ad, r.T, rot, r.q, r.k, qo, ko, lens=r.lens_d, starts=r.starts)
    before = r.qkv.clone()
    bdssm.rotary_step(r.ad, r.T, rot, r.q, r.k, r.q, r.k, lens=r.lens_d, starts=r.starts)
    assert torch.equal(r.q, qo) and torch.equal(r.k, ko)
    w = (r.H + r.KV) * r.D
    assert torch.equal(r.qkv[:, w:], before[:, w:])
    # one of the two alone; outputs with strides of their own
    wide = torch.zeros((r.n, r.H * r.D + 32), dtype=r.td, device="cuda")
    q0 = before[:, :r.H * r.D].view(r.n, r.H, r.D)
    bdssm.rotary_step(r.ad, r.T, rot, q0, None, wide[:, 16:16 + r.H * r.D].view(r.n, r.H, r.D), None, lens=r.lens_d,
                      starts=r.starts)
    assert torch.equal(wide[:, 16:16 + r.H * r.D].view(r.n, r.H, r.D), qo) and not wide[:, :16].any()
    k1 = torch.empty_like(ko)
    bdssm.rotary_step(r.ad, r.T, rot, None, before[:, r.H * r.D:w].view(r.n, r.KV, r.D), None, k1, lens=r.lens_d,
                      starts=r.starts)
    assert torch.equal(k1, ko)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("dim,interleaved", [(64, False), (48, True), (50, False)])
def test_append_is_the_step_and_the_append(dtype, page, dim, interleaved):
    import torch
    _case(f"rotary append page {page} dim {dim} dtype {dtype}")
    mk = lambda: Rows([page - 1, 0, 3 * page + 5, 40], [33, 0, 1, 2 * page + 3], dtype=dtype, page=page)  # noqa: E731
    r, s = mk(), mk()
    for x in (r, s):
        x.table[3, 1] = -1       # tokens of a page that is not held are dropped
        x.table[0, 1] = 10000
    rot = bdssm.Rotary(bdssm.rotary_turns(dim), interleaved, 0.5)
    qo, ko, q2, k2 = (torch.full((r.n, h, r.D), 9.0, dtype=r.td, device="cuda") for h in (r.H, r.KV, r.H, r.KV))
    l1, l2 = torch.zeros_like(r.lens_d), torch.zeros_like(r.lens_d)
    bdssm.rotary_append(r.ad, r.T, rot, r.q, r.k, r.v, r.cache(), qo, ko, l1, starts=r.starts)
    bdssm.rotary_step(s.ad, s.T, rot, s.q, s.k, q2, k2, lens=s.lens_d, starts=s.starts)
    bdssm.kv_append(s.ad, s.T, k2, s.v, s.cache(), l2, starts=s.starts)
    for a, b in ((qo, q2), (ko, k2), (r.kp, s.kp), (r.vp, s.vp), (l1, l2)):
        assert torch.equal(a, b)
    near(qo, *turned(_np(r.q), r.pos, frequencies(dim), interleaved, 0.5), dtype, "q")
    # keys alone, and keys in place
    t = mk()
    t.table[3, 1], t.table[0, 1] = -1, 10000
    bdssm.rotary_append(t.ad, t.T, rot, None, t.k, t.v, t.cache(), None, t.k, None, starts=t.starts)
    assert torch.equal(t.kp, s.kp) and torch.equal(t.vp, s.vp) and torch.equal(t.k, k2)


def test_append_past_the_table_and_with_positions():
    import torch
    _case("rotary append past the table")
    r = Rows([10, 30], [20, 20], page=16)
    r.table = r.table[:, :3].contiguous()  # 48 slots
    pos = torch.arange(100, 140, dtype=torch.int32, device="cuda")
    rot = bdssm.Rotary(bdssm.rotary_turns(64), positions=pos)
    qo, lens_out = torch.empty_like(r.q), torch.zeros_like(r.lens_d)
    bdssm.rotary_append(r.ad, r.T, rot, r.q, r.k, r.v, r.cache(), qo, None, lens_out, starts=r.starts)
    assert lens_out.tolist() == [30, 48]
    f = frequencies(64)
    near(qo, *turned(_np(r.q), np.arange(100, 140), f, False, 1.0), BF16, "q")
    want, tol = turned(_np(r.k), np.arange(100, 140), f, False, 1.0)
    for b, L in enumerate((10, 30)):
        for i in range(20):
            j = L + i
            if j >= 48:
                continue
            got = r.kp[r.table[b, j // 16], :, j % 16]
            near(got, want[20 * b + i], tol[20 * b + i], BF16, "key")
            assert torch.equal(r.vp[r.table[b, j // 16], :, j % 16], r.v[20 * b + i])


def test_rows_past_a_stream_stay():
    import torch
    _case("rotary rows past the last")
    r = Rows([5, 5], [30, 12])
    starts = torch.tensor([0, 25, 34], dtype=torch.int32, device="cuda")  # rows 34 on belong to no stream
    rot = bdssm.Rotary(bdssm.rotary_turns(64))
    qo, ko = (torch.full((r.n, h, r.D), 9.0, dtype=r.td, device="cuda") for h in (r.H, r.KV))
    bdssm.rotary_step(r.ad, 20, rot, r.q, r.k, qo, ko, lens=r.lens_d, starts=starts)  # 20 of the first stream's 25
    assert (qo[20:25] == 9).all() and (qo[34:] == 9).all() and (ko[34:] == 9).all()
    pos = np.concatenate([np.arange(5, 25), np.arange(5, 14)])
    rows = list(range(20)) + list(range(25, 34))
    near(qo[rows], *turned(_np(r.q[rows]), pos, frequencies(64), False, 1.0), BF16, "q")


def test_graph_and_stream():
    import torch
    _case("rotary graph")
    r = Rows([40, 7], [32, 32], ragged=False)
    rot = bdssm.Rotary(bdssm.rotary_turns(64))
    qo, lens_out = torch.empty_like(r.q), torch.zeros_like(r.lens_d)
    cache = r.cache()
    call = lambda: bdssm.rotary_append(r.ad, r.T, rot, r.q, r.k, r.v, cache, qo, None, lens_out)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([40, 7], [0, 1], [33, 16]):
        r.lens_d.copy_(torch.tensor(lens, dtype=torch.int32))
        r.kp.fill_(0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        bdssm.rotary_append(r.ad, r.T, rot, r.q, r.k, r.v, cache, qo, None, lens_out, stream=side)
        side.synchronize()
        want, pages = qo.clone(), r.kp.clone()
        qo.fill_(0)
        r.kp.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, want) and torch.equal(r.kp, pages) and lens_out.tolist() == [x + 32 for x in lens]
