"""Argument checks of the norm and attention calls, on the CPU: every refusal happens before
anything is launched."""
import ctypes

import pytest

from bidirectional_mamba_state_amd import bdssm

BASE = 1 << 40
GB = 1 << 30
SIZE_MAX = ctypes.c_size_t(-1).value


def gated(nd=None, y=BASE, z=BASE + GB, zs=None, w=BASE + 2 * GB, first=0, out=BASE + 3 * GB, **kw):
    d = dict(rows=8, width=100, dtype=bdssm.BF16, groups=2, x_dtype=bdssm.F32)
    d.update(kw)
    nd = bdssm.norm_dims(**d) if nd is None else nd
    return bdssm.load().bdssm_gated_norm(ctypes.byref(nd), y, z, nd.width if zs is None else zs, w, first, out, None)


def test_gated_norm_refusals():
    lib = bdssm.load()
    assert lib.bdssm_gated_norm(None, BASE, BASE, 1, None, 0, BASE, None) == bdssm.ERR_NULL
    assert gated(y=None) == gated(z=None) == gated(out=None) == bdssm.ERR_NULL
    assert gated(groups=3) == gated(rows=-1) == gated(width=0) == gated(groups=0) == bdssm.ERR_SHAPE
    assert gated(zs=99) == bdssm.ERR_SHAPE
    assert gated(dtype=2) == gated(dtype=bdssm.F32, x_dtype=bdssm.BF16) == bdssm.ERR_UNSUPPORTED
    assert gated(eps=0.0) == gated(eps=float("nan")) == gated(kind=bdssm.NORM_LAYER) == bdssm.ERR_UNSUPPORTED
    assert gated(first=2) == gated(width=16385, groups=1) == gated(rows=1 << 31) == bdssm.ERR_UNSUPPORTED
    assert gated(z=BASE + GB + 1) == gated(y=BASE + 2) == gated(w=BASE + 2 * GB + 2) == bdssm.ERR_ALIGN
    assert gated(out=BASE + GB + 50) == gated(out=BASE + 3196) == gated(out=BASE + 2 * GB) == bdssm.ERR_ALIAS
    assert gated(out=BASE) == bdssm.ERR_ALIAS                              # y itself, but another type
    assert gated(rows=0) == bdssm.OK


def residual(x=BASE, o=BASE + GB, pw=None, w=BASE + 2 * GB, gate=None, gain=None, shift=None, ms=0, scale=1.0,
             x_out=BASE + 4 * GB, u=BASE + 5 * GB, **kw):
    d = dict(rows=8, width=100, dtype=bdssm.BF16, x_dtype=bdssm.F32, rows_per_stream=3)
    d.update(kw)
    nd = bdssm.norm_dims(**d)
    r = bdssm.Residual(x, o, pw, w, gate, gain, shift, ms, scale)
    return bdssm.load().bdssm_residual_norm(ctypes.byref(nd), ctypes.byref(r), x_out, u, None)


def test_residual_norm_refusals():
    lib = bdssm.load()
    nd = bdssm.norm_dims(8, 100, bdssm.BF16)
    assert lib.bdssm_residual_norm(ctypes.byref(nd), None, BASE, BASE, None) == bdssm.ERR_NULL
    assert residual(x=None) == residual(x_out=None, u=None) == bdssm.ERR_NULL
    assert residual(groups=2) == residual(gate=BASE + 6 * GB, ms=99) == bdssm.ERR_SHAPE
    assert residual(gain=BASE + 6 * GB, ms=100, rows_per_stream=0) == bdssm.ERR_SHAPE
    assert residual(width=16385) == residual(kind=2) == bdssm.ERR_UNSUPPORTED
    assert residual(o=BASE + GB + 1) == residual(w=BASE + 2 * GB + 2) == residual(x_out=BASE + 2) == bdssm.ERR_ALIGN
    assert residual(x_out=BASE + 64) == residual(u=BASE) == residual(u=BASE + 4 * GB) == bdssm.ERR_ALIAS
    # gate of three streams (8 rows by 3): its last row's end
    last = BASE + 6 * GB + 2 * 200 * 2 + 99 * 2
    assert residual(gate=BASE + 6 * GB, ms=200, u=last) == bdssm.ERR_ALIAS
    assert residual(rows=0) == bdssm.OK


class Chunk:
    def __init__(self, **kw):
        d = dict(q=BASE, k=BASE + GB, v=BASE + 2 * GB, q_stride=4 * 64, k_stride=2 * 64, v_stride=2 * 64, tokens=16,
                 starts=None, block_len=8)
        d.update(kw)
        self.s = bdssm.AttnChunk(*[d[n] for n in ("q", "k", "v", "q_stride", "k_stride", "v_stride", "tokens", "starts",
                                                  "block_len")])


class Cache:
    def __init__(self, **kw):
        d = dict(k=BASE + 3 * GB, v=BASE + 4 * GB, table=BASE + 5 * GB, lens=BASE + 6 * GB, num_pages=10, max_pages=4,
                 max_len=64)
        d.update(kw)
        self.s = bdssm.KvCachePtrs(*[d[n] for n in ("k", "v", "table", "lens", "num_pages", "max_pages", "max_len")])


def dims(batch=2, nheads=4, kv_heads=2, headdim=64, dtype=bdssm.BF16, page=16):
    return bdssm.attn_dims(batch, nheads, kv_heads, headdim, dtype, page)


def step(d=None, ch=None, ca=None, m=(0.125, 0, 0, 0), out=BASE + 8 * GB, ws=BASE + 9 * GB, wsb=GB):
    d, ch, ca = d or dims(), ch or Chunk(), ca or Cache()
    mask = bdssm.AttnMask(*m)
    return bdssm.load().bdssm_attn_step(ctypes.byref(d), ctypes.byref(ch.s), ctypes.byref(ca.s), ctypes.byref(mask), out,
                                        ws, wsb, None)


def append(d=None, ch=None, ca=None, lens_out=BASE + 8 * GB):
    d, ch, ca = d or dims(), ch or Chunk(q=None, q_stride=0), ca or Cache()
    return bdssm.load().bdssm_kv_append(ctypes.byref(d), ctypes.byref(ch.s), ctypes.byref(ca.s), lens_out, None)


BAD = [  # dims, chunk, cache -> status, for both calls
    (dict(nheads=3), {}, {}, bdssm.ERR_SHAPE), (dict(kv_heads=0), {}, {}, bdssm.ERR_SHAPE),
    (dict(batch=-1), {}, {}, bdssm.ERR_SHAPE), (dict(headdim=80), {}, {}, bdssm.ERR_UNSUPPORTED),
    (dict(page=24), {}, {}, bdssm.ERR_UNSUPPORTED), (dict(dtype=3), {}, {}, bdssm.ERR_UNSUPPORTED),
    ({}, dict(block_len=-1), {}, bdssm.ERR_SHAPE), ({}, dict(tokens=17), {}, bdssm.ERR_SHAPE),
    ({}, dict(k_stride=127), {}, bdssm.ERR_SHAPE), ({}, dict(k=None), {}, bdssm.ERR_NULL),
    ({}, dict(v=None), {}, bdssm.ERR_NULL), ({}, dict(v=BASE + 8), {}, bdssm.ERR_ALIGN),
    ({}, dict(v_stride=132), {}, bdssm.ERR_ALIGN), ({}, dict(starts=BASE + 7 * GB + 2), {}, bdssm.ERR_ALIGN),
    ({}, {}, dict(k=None), bdssm.ERR_NULL), ({}, {}, dict(table=None), bdssm.ERR_NULL),
    ({}, {}, dict(lens=None), bdssm.ERR_NULL), ({}, {}, dict(max_len=65), bdssm.ERR_SHAPE),
    ({}, {}, dict(num_pages=-1), bdssm.ERR_SHAPE), ({}, {}, dict(v=BASE + 4 * GB + 8), bdssm.ERR_ALIGN),
    ({}, {}, dict(lens=BASE + 6 * GB + 1), bdssm.ERR_ALIGN),
    ({}, {}, dict(max_pages=1 << 28, max_len=(1 << 31) - 1), bdssm.ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("d,ch,ca,want", BAD)
def test_shared_refusals(d, ch, ca, want):
    assert step(dims(**d), Chunk(**ch), Cache(**ca)) == want
    assert append(dims(**d), Chunk(**{**dict(q=None, q_stride=0), **ch}), Cache(**ca)) == want


def test_attn_step_refusals():
    lib = bdssm.load()
    d, ch, ca, m = dims(), Chunk().s, Cache().s, bdssm.AttnMask(0.125, 0, 0, 0)
    r = ctypes.byref
    assert lib.bdssm_attn_step(None, r(ch), r(ca), r(m), BASE, None, 0, None) == bdssm.ERR_NULL
    assert lib.bdssm_attn_step(r(d), None, r(ca), r(m), BASE, None, 0, None) == bdssm.ERR_NULL
    assert lib.bdssm_attn_step(r(d), r(ch), None, r(m), BASE, None, 0, None) == bdssm.ERR_NULL
    assert lib.bdssm_attn_step(r(d), r(ch), r(ca), None, BASE, None, 0, None) == bdssm.ERR_NULL
    assert step(out=None) == step(ch=Chunk(q=None)) == bdssm.ERR_NULL
    assert step(m=(0.1, -1, 0, 0)) == step(m=(0.1, 0, -1, 0)) == step(m=(0.1, 0, 0, -1)) == bdssm.ERR_SHAPE
    assert step(m=(float("inf"), 0, 0, 0)) == step(m=(float("nan"), 0, 0, 0)) == bdssm.ERR_UNSUPPORTED
    assert step(ch=Chunk(q_stride=255)) == bdssm.ERR_SHAPE
    assert step(ch=Chunk(q=BASE + 4)) == step(ch=Chunk(q_stride=260)) == step(out=BASE + 8 * GB + 8) == bdssm.ERR_ALIGN
    rows = 15 * 4 * 64 * 2  # the last row's first byte
    for on in (BASE + rows, BASE + GB, BASE + 2 * GB, BASE + 3 * GB, BASE + 4 * GB, BASE + 5 * GB, BASE + 6 * GB):
        assert step(out=on) == bdssm.ERR_ALIAS
    assert step(ch=Chunk(tokens=0, block_len=0)) == bdssm.OK
    assert step(d=dims(batch=0), ch=Chunk(tokens=0)) == bdssm.OK
    ws = bdssm.attn_step_workspace
    mask = bdssm.attn_mask(0.1)
    assert ws(dims(headdim=80), 8, 64, mask) == ws(dims(), -1, 64, mask) == ws(dims(), 8, -1, mask) == SIZE_MAX
    assert ws(dims(), 8, 64, bdssm.attn_mask(0.1, window=-1)) == SIZE_MAX


def test_kv_append_refusals():
    assert append(lens_out=BASE + 8 * GB + 2) == bdssm.ERR_ALIGN
    assert append(lens_out=BASE + 6 * GB) == append(lens_out=BASE + 5 * GB) == bdssm.ERR_ALIAS
    assert append(ca=Cache(v=BASE + 3 * GB + 4096)) == bdssm.ERR_ALIAS          # pools on each other
    assert append(ca=Cache(k=BASE + GB)) == bdssm.ERR_ALIAS                     # pool on the chunk
    assert append(d=dims(batch=0), ch=Chunk(tokens=0, q=None)) == bdssm.OK


def test_binding_checks_shapes_and_types():
    torch = pytest.importorskip("torch")
    nd = bdssm.norm_dims(4, 8, bdssm.F32)
    t = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        bdssm.gated_norm(nd, t, t, None, t)
    with pytest.raises(ValueError):
        bdssm.KvCache(dims(), torch.zeros(3, 2, 16, 64), torch.zeros(3, 2, 16, 64), None, None, 0)
    with pytest.raises(ValueError):
        bdssm._rows(FakeCuda(torch.zeros(4, 2, 64).transpose(1, 2)), "q", torch.float32, (4, 64, 2))
    assert bdssm._rows(FakeCuda(torch.zeros(4, 200)[:, 8:136].view(4, 2, 64)), "q", torch.float32, (4, 2, 64))[1] == 200


class FakeCuda:
    """A host tensor that claims to be a device one, for checks that never read memory."""
    is_cuda = True

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)
