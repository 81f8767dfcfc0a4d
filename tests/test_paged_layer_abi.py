"""Argument checks of the rotary, scored-attention and page calls, on the CPU: every refusal happens
before anything is launched. And the table of rotary frequencies, which the host makes."""
import ctypes

import numpy as np
import pytest

from bidirectional_mamba_state_amd import bdssm
from test_layer_ops_abi import BAD, BASE, GB, SIZE_MAX, Cache, Chunk, FakeCuda, dims

r = ctypes.byref
NULL, SHAPE, UNSUPPORTED, ALIGN, ALIAS, WORKSPACE = (bdssm.ERR_NULL, bdssm.ERR_SHAPE, bdssm.ERR_UNSUPPORTED, bdssm.ERR_ALIGN,
                                                     bdssm.ERR_ALIAS, bdssm.ERR_WORKSPACE)


# ------------------------------------------------------------------------------ attention
def scores(cap=0.0, slopes=None, prefix=None, first=None, last=None):
    return bdssm.AttnScoresPtrs(cap, slopes, prefix, first, last)


def step_ex(d=None, ch=None, ca=None, m=(0.125, 0, 0, 0), s=None, out=BASE + 8 * GB, ws=BASE + 9 * GB, wsb=GB):
    d, ch, ca, s = d or dims(), ch or Chunk(), ca or Cache(), s or scores()
    return bdssm.load().bdssm_attn_step_ex(r(d), r(ch.s), r(ca.s), r(bdssm.AttnMask(*m)), r(s), out, ws, wsb, None)


@pytest.mark.parametrize("d,ch,ca,want", BAD)
def test_attn_step_ex_shares_the_steps_refusals(d, ch, ca, want):
    assert step_ex(dims(**d), Chunk(**ch), Cache(**ca)) == want


def test_attn_step_ex_refusals():
    lib = bdssm.load()
    d, ch, ca, m = dims(), Chunk().s, Cache().s, bdssm.AttnMask(0.125, 0, 0, 0)
    assert lib.bdssm_attn_step_ex(r(d), r(ch), r(ca), r(m), None, BASE, None, 0, None) == NULL
    assert lib.bdssm_attn_step_ex(r(d), r(ch), r(ca), None, r(scores()), BASE, None, 0, None) == NULL
    assert step_ex(out=None) == NULL
    for cap in (-1.0, float("nan"), float("inf"), -float("inf"), 1e-39, 2e38):
        assert step_ex(s=scores(cap)) == UNSUPPORTED, cap
    assert step_ex(s=scores(1e-37), m=(10.0, 0, 0, 0)) == UNSUPPORTED  # scale / cap is infinite
    at = BASE + 10 * GB
    for scale in (2.0**-65, 2.0**65):
        assert step_ex(s=scores(slopes=at), m=(scale, 0, 0, 0)) == UNSUPPORTED
    for name in ("slopes", "prefix", "first", "last"):
        assert step_ex(s=scores(**{name: at + 2})) == ALIGN
        size = dict(slopes=4, prefix=2, first=16, last=16)[name] * 4
        assert step_ex(s=scores(**{name: BASE + 8 * GB + 64})) == ALIAS             # inside out
        assert step_ex(s=scores(**{name: BASE + 8 * GB - size + 4})) == ALIAS       # its last entry
    # the workspace on a range, where the plan needs one
    ca = Cache(max_pages=100000, max_len=1000000)
    assert step_ex(ca=ca, ws=None) == WORKSPACE
    assert step_ex(ca=ca, s=scores(first=BASE + 9 * GB + 64)) == ALIAS
    assert step_ex(ch=Chunk(tokens=0, block_len=0)) == bdssm.OK
    assert step_ex(d=dims(batch=0), ch=Chunk(tokens=0)) == bdssm.OK
    ws = lambda d, T, L, m, s: bdssm.load().bdssm_attn_step_ex_workspace(r(d), T, L, r(m), r(s))  # noqa: E731
    mask = bdssm.attn_mask(0.1)
    assert ws(dims(), 8, 64, mask, scores(-1.0)) == ws(dims(headdim=80), 8, 64, mask, scores()) == SIZE_MAX
    for T, L in ((1, 100000), (32, 5000), (700, 700)):
        assert ws(dims(), T, L, mask, scores(5.0)) == bdssm.attn_step_workspace(dims(), T, L, mask)
    assert lib.bdssm_attn_step_ex_workspace(r(d), 8, 64, r(mask), None) == SIZE_MAX


# --------------------------------------------------------------------------------- rotary
def rotary(dim=64, interleaved=0, scale=1.0, turns=BASE + 11 * GB, positions=None):
    return bdssm.RotaryPtrs(dim, interleaved, scale, turns, positions)


def rout(q=BASE + 12 * GB, k=BASE + 13 * GB, qs=256, ks=128):
    return bdssm.RotaryOut(q, k, qs, ks)


def rstep(d=None, ch=None, ro=None, lens=BASE + 6 * GB, out=None):
    d, ch, ro, out = d or dims(), ch or Chunk(), ro or rotary(), out or rout()
    return bdssm.load().bdssm_rotary_step(r(d), r(ch.s), r(ro), lens, r(out), None)


def rappend(d=None, ch=None, ca=None, ro=None, out=None, lens_out=BASE + 14 * GB):
    d, ch, ca, ro, out = d or dims(), ch or Chunk(), ca or Cache(), ro or rotary(), out or rout()
    return bdssm.load().bdssm_rotary_append(r(d), r(ch.s), r(ca.s), r(ro), r(out), lens_out, None)


BOTH = [  # chunk, rotary, out -> status, for the step and the append
    ({}, dict(dim=0), {}, SHAPE), ({}, dict(dim=7), {}, SHAPE), ({}, dict(dim=66), {}, SHAPE), ({}, dict(dim=-2), {}, SHAPE),
    ({}, dict(interleaved=2), {}, UNSUPPORTED), ({}, dict(interleaved=-1), {}, UNSUPPORTED),
    ({}, dict(scale=float("nan")), {}, UNSUPPORTED), ({}, dict(scale=float("inf")), {}, UNSUPPORTED),
    ({}, dict(turns=None), {}, NULL), ({}, dict(turns=BASE + 11 * GB + 4), {}, ALIGN),
    ({}, dict(positions=BASE + 15 * GB + 2), {}, ALIGN),
    ({}, {}, dict(q=None), NULL), (dict(q=None), {}, {}, NULL),
    ({}, {}, dict(qs=255), SHAPE), ({}, {}, dict(ks=127), SHAPE), ({}, {}, dict(qs=260), ALIGN), ({}, {}, dict(ks=132), ALIGN),
    ({}, {}, dict(q=BASE + 12 * GB + 8), ALIGN), ({}, {}, dict(k=BASE + 13 * GB + 4), ALIGN),
    ({}, {}, dict(qs=(1 << 24) + 8), UNSUPPORTED), ({}, {}, dict(ks=(1 << 24) + 8), UNSUPPORTED),
    ({}, {}, dict(q=BASE + 16), ALIAS),                      # q, moved
    ({}, {}, dict(q=BASE, qs=512), ALIAS),                   # q, other stride
    ({}, {}, dict(q=BASE + GB), ALIAS), ({}, {}, dict(k=BASE), ALIAS),  # each on the other's input
    ({}, {}, dict(k=BASE + 12 * GB + 128), ALIAS),           # outputs on each other
    ({}, {}, dict(q=BASE + 11 * GB - 64), ALIAS),            # on the table of turns
    ({}, dict(positions=BASE + 13 * GB + 64), {}, ALIAS),
    ({}, {}, dict(k=BASE + 6 * GB - 256), ALIAS),            # on lens
]


@pytest.mark.parametrize("ch,ro,out,want", BOTH)
def test_rotary_refusals_of_both(ch, ro, out, want):
    assert rstep(ch=Chunk(**ch), ro=rotary(**ro), out=rout(**out)) == want
    assert rappend(ch=Chunk(**ch), ro=rotary(**ro), out=rout(**out)) == want


def test_rotary_step_refusals():
    lib = bdssm.load()
    d, ch, ro, out = dims(), Chunk().s, rotary(), rout()
    assert lib.bdssm_rotary_step(None, r(ch), r(ro), None, r(out), None) == NULL
    assert lib.bdssm_rotary_step(r(d), None, r(ro), None, r(out), None) == NULL
    assert lib.bdssm_rotary_step(r(d), r(ch), None, None, r(out), None) == NULL
    assert lib.bdssm_rotary_step(r(d), r(ch), r(ro), None, None, None) == NULL
    assert rstep(out=rout(k=None)) == rstep(ch=Chunk(k=None)) == rstep(ch=Chunk(q=None, k=None), out=rout(q=None, k=None)) == NULL
    assert rstep(ch=Chunk(tokens=17)) == rstep(ch=Chunk(block_len=-1)) == rstep(ch=Chunk(q_stride=255)) == SHAPE
    assert rstep(d=dims(headdim=80)) == rstep(ch=Chunk(k_stride=(1 << 24) + 8)) == UNSUPPORTED
    far = (1 << 24) + 1  # tokens of a stream
    assert rstep(ch=Chunk(tokens=2 * far, block_len=far, k=BASE + 100 * GB), out=rout(BASE + 200 * GB, BASE + 300 * GB)) == UNSUPPORTED
    assert rstep(ch=Chunk(q=BASE + 4)) == rstep(ch=Chunk(k_stride=132)) == rstep(lens=BASE + 2) == ALIGN
    assert rstep(ch=Chunk(tokens=0, block_len=0)) == rstep(d=dims(batch=0), ch=Chunk(tokens=0)) == bdssm.OK
    # slices of one projection: in place, and each beside the other, is no overlap; half a row off is
    slices = dict(q=BASE, k=BASE + 512, v=BASE + 768, q_stride=512, k_stride=512, v_stride=512, tokens=0, block_len=0)
    assert rstep(ch=Chunk(**slices), out=rout(BASE, BASE + 512, 512, 512)) == bdssm.OK
    slices.update(tokens=16, block_len=8)
    assert rstep(ch=Chunk(**slices), out=rout(BASE, BASE + 256, 512, 512)) == ALIAS
    assert rstep(ch=Chunk(**slices), out=rout(BASE + 512, BASE, 512, 512)) == ALIAS
    # queries that reach 384 bytes into the next row, where its keys begin at 256
    slices.update(q=BASE + 1024 - 128, k=BASE + 256)
    assert rstep(ch=Chunk(**slices), out=rout(BASE + 1024 - 128, BASE + 256, 512, 512)) == ALIAS


def test_rotary_append_refusals():
    lib = bdssm.load()
    d, ch, ca, ro, out = dims(), Chunk().s, Cache().s, rotary(), rout()
    assert lib.bdssm_rotary_append(None, r(ch), r(ca), r(ro), r(out), None, None) == NULL
    assert lib.bdssm_rotary_append(r(d), None, r(ca), r(ro), r(out), None, None) == NULL
    assert lib.bdssm_rotary_append(r(d), r(ch), None, r(ro), r(out), None, None) == NULL
    assert lib.bdssm_rotary_append(r(d), r(ch), r(ca), None, r(out), None, None) == NULL
    assert lib.bdssm_rotary_append(r(d), r(ch), r(ca), r(ro), None, None, None) == NULL  # there are queries
    assert rappend(ch=Chunk(k=None)) == rappend(ch=Chunk(v=None)) == NULL
    assert rappend(lens_out=BASE + 2) == ALIGN
    assert rappend(lens_out=BASE + 6 * GB) == rappend(lens_out=BASE + 5 * GB) == rappend(lens_out=BASE + 12 * GB + 64) == ALIAS
    assert rappend(out=rout(q=BASE + 3 * GB)) == rappend(out=rout(k=BASE + 4 * GB)) == rappend(out=rout(k=BASE + 2 * GB)) == ALIAS
    assert rappend(ca=Cache(v=BASE + 3 * GB + 4096)) == rappend(ca=Cache(k=BASE + GB)) == ALIAS
    assert rappend(d=dims(batch=0), ch=Chunk(tokens=0)) == bdssm.OK


@pytest.mark.parametrize("d,ch,ca,want", BAD)
def test_rotary_append_shares_the_appends_refusals(d, ch, ca, want):
    assert rappend(dims(**d), Chunk(**ch), Cache(**ca)) == want


def freqs(dim=64, kind=bdssm.ROTARY_PLAIN, base=1e4, factor=4.0, trained=4096, low=1.0, high=32.0):
    out = np.zeros(300, dtype=np.uint64)
    rc = bdssm.load().bdssm_rotary_turns(r(bdssm.RotaryFreqs(dim, kind, base, factor, trained, low, high)), out.ctypes.data)
    return rc, out[:max(dim, 0) // 2]


def test_rotary_turns_refusals():
    lib = bdssm.load()
    f = bdssm.RotaryFreqs(64, 0, 1e4, 1.0, 0, 1.0, 2.0)
    assert lib.bdssm_rotary_turns(None, BASE) == lib.bdssm_rotary_turns(r(f), None) == NULL
    for dim in (0, 1, 7, -2, 514):
        assert freqs(dim)[0] == SHAPE
    nan, inf = float("nan"), float("inf")
    for bad in (dict(kind=4), dict(kind=-1), dict(base=0.5), dict(base=nan), dict(base=inf), dict(kind=1, factor=0.0),
                dict(kind=1, factor=-2.0), dict(kind=1, factor=nan), dict(kind=2, factor=inf), dict(kind=2, dim=2),
                dict(kind=3, trained=0), dict(kind=3, low=4.0, high=4.0), dict(kind=3, low=nan), dict(kind=3, high=inf)):
        assert freqs(**bad)[0] == UNSUPPORTED, bad
    assert freqs(kind=bdssm.ROTARY_PLAIN, factor=0.0)[0] == bdssm.OK  # not looked at


@pytest.mark.parametrize("kind,more", [(0, {}), (1, dict(factor=4.0)), (2, dict(factor=8.0)),
                                       (3, dict(factor=32.0, trained=8192, low=1.0, high=4.0)),
                                       (3, dict(factor=16.0, trained=4096, low=1.0, high=32.0)), (1, dict(factor=0.01))])
@pytest.mark.parametrize("dim", [2, 6, 64, 128, 512])
def test_rotary_turns(kind, more, dim):
    """Against the formulas in 80-bit floats, in radians: within 2^-60 of the frequency."""
    if kind == 2 and dim == 2:
        return
    ld = np.longdouble
    base = ld(500000.0)
    rc, got = freqs(dim=dim, kind=kind, base=500000.0, **more)
    assert rc == bdssm.OK
    s = ld(more.get("factor", 1.0))
    if kind == 2:
        base *= s ** (ld(dim) / ld(dim - 2))
    pi2 = 2 * ld("3.14159265358979323846264338327950288")
    f = np.exp(-2 * np.arange(dim // 2, dtype=ld) / ld(dim) * np.log(base))
    if kind == 1:
        f = f / s
    if kind == 3:
        g = np.clip((more["trained"] * f / pi2 - more["low"]) / (ld(more["high"]) - more["low"]), 0, 1)
        assert (g == 0).any() or dim < 64
        f = f * (g + (1 - g) / s)
    turns = f / pi2
    back = np.array([ld(int(x) >> 32) * ld(2) ** -32 + ld(int(x) & 0xffffffff) * ld(2) ** -64 for x in got])
    assert np.all(np.abs(back - (turns - np.floor(turns))) <= turns * ld(2) ** -58 + ld(2) ** -62)


# ---------------------------------------------------------------------------------- pages
def pd(batch=2, page=16, P=100, per=8):
    return bdssm.page_dims(batch, page, P, per)


def pages(table=BASE, lens=BASE + GB, uses=BASE + 2 * GB):
    return bdssm.PagesPtrs(table, lens, uses)


OUT = dict(t=BASE + 3 * GB, u=BASE + 4 * GB, n=BASE + 5 * GB, ws=BASE + 6 * GB, wsb=GB)


def advance(d=None, g=None, starts=None, T=8, window=0, sinks=0, **kw):
    o = {**OUT, **kw}
    return bdssm.load().bdssm_pages_advance(r(d or pd()), r(g or pages()), starts, T, window, sinks, o["t"], o["u"], o["n"],
                                            o["ws"], o["wsb"], None)


def fork(d=None, g=None, parents=BASE + 7 * GB, lens=BASE + 8 * GB, copies=BASE + 9 * GB, **kw):
    o = {**OUT, **kw}
    return bdssm.load().bdssm_pages_fork(r(d or pd()), r(g or pages()), parents, o["t"], lens, o["u"], copies, o["n"],
                                         o["ws"], o["wsb"], None)


def compact(d=None, g=None, copies=BASE + 9 * GB, **kw):
    o = {**OUT, **kw}
    return bdssm.load().bdssm_pages_compact(r(d or pd()), r(g or pages()), o["t"], o["u"], copies, o["n"], o["ws"], o["wsb"],
                                            None)


@pytest.mark.parametrize("call", [advance, fork, compact])
def test_pages_refusals_of_all(call):
    assert call(d=pd(batch=-1)) == call(d=pd(P=-1)) == call(d=pd(per=-1)) == SHAPE
    assert call(d=pd(page=24)) == call(d=pd(batch=65536)) == call(d=pd(per=(1 << 27) + 1)) == UNSUPPORTED
    assert call(g=pages(table=None)) == call(g=pages(lens=None)) == call(g=pages(uses=None)) == NULL
    assert call(t=None) == call(u=None) == call(n=None) == NULL
    assert call(g=pages(table=BASE + 2)) == call(g=pages(lens=BASE + GB + 1)) == call(u=BASE + 4 * GB + 2) == ALIGN
    assert call(ws=BASE + 6 * GB + 8) == call(n=BASE + 5 * GB + 1) == ALIGN
    need = bdssm.pages_workspace(pd())
    assert call(ws=None) == call(wsb=need - 1) == WORKSPACE
    assert call(ws=BASE + 4) == ALIGN
    assert call(t=BASE + 4) == call(u=BASE + 2 * GB + 4) == call(t=BASE + 2 * GB) == call(u=BASE) == ALIAS
    assert call(n=BASE + GB + 4) == call(n=BASE + 3 * GB) == call(t=BASE + 4 * GB) == ALIAS
    assert call(ws=BASE) == call(ws=BASE + 2 * GB - need + 16) == call(ws=BASE + 3 * GB) == call(ws=BASE + 5 * GB) == ALIAS


def test_pages_refusals_of_each():
    lib = bdssm.load()
    assert lib.bdssm_pages_advance(None, r(pages()), None, 1, 0, 0, *[BASE] * 4, GB, None) == NULL
    assert lib.bdssm_pages_advance(r(pd()), None, None, 1, 0, 0, *[BASE] * 4, GB, None) == NULL
    assert advance(T=-1) == advance(window=-1) == advance(sinks=-1) == SHAPE
    assert advance(starts=BASE + 10 * GB + 2) == ALIGN
    # 2^16 - 1 streams that could each need 2^15 + 1 pages
    far = dict(g=pages(BASE, BASE + 16384 * GB, BASE + 16385 * GB), t=BASE, u=BASE + 16386 * GB, n=BASE + 16387 * GB,
               ws=BASE + 16388 * GB)
    assert advance(d=pd(batch=65535, per=1 << 16), T=16 << 15, **far) == UNSUPPORTED
    assert advance(starts=BASE + 3 * GB + 4) == advance(starts=BASE + 6 * GB) == ALIAS
    assert fork(parents=None) == fork(lens=None) == fork(copies=None) == NULL
    assert fork(t=BASE) == fork(lens=BASE + GB) == fork(lens=BASE + 7 * GB) == fork(copies=BASE + 8 * GB - 8) == ALIAS
    assert fork(parents=BASE + 7 * GB + 2) == fork(copies=BASE + 9 * GB + 1) == ALIGN
    assert compact(copies=None) == NULL
    assert compact(copies=BASE + 3 * GB - 4) == ALIAS
    assert bdssm.pages_workspace(pd(page=24)) == SIZE_MAX
    assert lib.bdssm_pages_workspace(None) == SIZE_MAX
    sizes = [bdssm.pages_workspace(pd(batch=b, P=p)) for b, p in ((0, 0), (1, 1), (2, 100), (64, 5000), (65535, 1 << 20))]
    assert sizes == sorted(sizes) and sizes[-1] < 1 << 24


def test_pages_copy_refusals():
    lib = bdssm.load()
    copy = lambda d=None, ca=None, c=BASE + 9 * GB, n=4: lib.bdssm_pages_copy(  # noqa: E731
        r(d or dims()), r((ca or Cache()).s), c, n, None)
    assert lib.bdssm_pages_copy(None, r(Cache().s), BASE, 1, None) == lib.bdssm_pages_copy(r(dims()), None, BASE, 1, None) == NULL
    assert copy(c=None) == copy(ca=Cache(k=None)) == copy(ca=Cache(v=None)) == NULL
    assert copy(n=-1) == copy(ca=Cache(num_pages=-1)) == SHAPE
    assert copy(d=dims(headdim=96)) == copy(d=dims(page=20)) == UNSUPPORTED
    assert copy(c=BASE + 9 * GB + 2) == copy(ca=Cache(k=BASE + 3 * GB + 8)) == ALIGN
    assert copy(c=BASE + 3 * GB + 64) == copy(c=BASE + 4 * GB - 28) == copy(ca=Cache(v=BASE + 3 * GB + 4096)) == ALIAS
    assert copy(n=0) == copy(n=0, c=None) == copy(ca=Cache(num_pages=0, k=None, v=None)) == bdssm.OK


def test_binding_checks_shapes_and_types():
    torch = pytest.importorskip("torch")
    ints = lambda *s: FakeCuda(torch.zeros(s, dtype=torch.int32))  # noqa: E731
    g = bdssm.Pages(pd(), ints(2, 8), ints(2), ints(100))
    for bad in ((ints(3, 8), ints(2), ints(100)), (ints(2, 8), ints(3), ints(100)), (ints(2, 8), ints(2), ints(99)),
                (FakeCuda(torch.zeros(2, 8)), ints(2), ints(100))):
        with pytest.raises(ValueError):
            bdssm.Pages(pd(), *bad)
    for t, u, n in ((ints(2, 7), ints(100), ints(1)), (ints(2, 8), ints(10), ints(1)), (ints(2, 8), ints(100), ints(2))):
        with pytest.raises(ValueError):
            bdssm.pages_advance(pd(), g, 1, t, u, n, None, stream=0)
    with pytest.raises(ValueError):
        bdssm.pages_fork(pd(), g, ints(3), ints(2, 8), ints(2), ints(100), ints(2, 2), ints(1), None, stream=0)
    with pytest.raises(ValueError):
        bdssm.pages_compact(pd(), g, ints(2, 8), ints(100), ints(49, 2), ints(1), None, stream=0)
    # bookkeeping and pools that were made for other sizes
    out = ints(3, 8), ints(100), ints(1)
    with pytest.raises(ValueError, match="made for"):
        bdssm.pages_advance(pd(batch=3), g, 1, *out, None, stream=0)
    with pytest.raises(ValueError, match="made for"):
        bdssm.pages_fork(pd(batch=3), g, ints(3), ints(3, 8), ints(3), ints(100), ints(3, 2), ints(1), None, stream=0)
    with pytest.raises(ValueError, match="made for"):
        bdssm.pages_compact(pd(P=101), g, ints(2, 8), ints(101), ints(50, 2), ints(1), None, stream=0)
    pool = FakeCuda(torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16))
    c = bdssm.KvCache(bdssm.attn_dims(2, 4, 2, 64, bdssm.BF16, 16), pool, pool, ints(2, 8), ints(2), 8)
    with pytest.raises(ValueError, match="its pages are"):
        bdssm.pages_copy(bdssm.attn_dims(2, 4, 2, 64, bdssm.BF16, 32), c, ints(1, 2), stream=0)
    with pytest.raises(ValueError):
        bdssm.AttnScores(slopes=ints(4))
    with pytest.raises(ValueError):
        bdssm.AttnScores(first=FakeCuda(torch.zeros(4)))
    with pytest.raises(ValueError):
        bdssm.Rotary(FakeCuda(torch.zeros(4)))
    with pytest.raises(TypeError):
        bdssm.Rotary(torch.zeros(4, dtype=torch.int64))
    rot = bdssm.Rotary(FakeCuda(torch.zeros(32, dtype=torch.int64)), positions=ints(5))
    bf = lambda *s: FakeCuda(torch.zeros(s, dtype=torch.bfloat16))  # noqa: E731
    with pytest.raises(ValueError):  # positions of other tokens
        bdssm.rotary_step(dims(), 8, rot, bf(16, 4, 64), None, bf(16, 4, 64), None, stream=0)
    with pytest.raises(ValueError):  # an output of another shape
        bdssm.rotary_step(dims(), 8, bdssm.Rotary(rot.turns), bf(16, 4, 64), None, bf(16, 2, 64), None, stream=0)
    s = bdssm.AttnScores(5.0, slopes=FakeCuda(torch.zeros(3)))
    with pytest.raises(ValueError):  # slopes of other heads
        bdssm.attn_step_ex(dims(), 8, bf(16, 4, 64), None, None, None, bdssm.attn_mask(1.0), s, bf(16, 4, 64), stream=0)
