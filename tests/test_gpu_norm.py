"""The norms around a layer (bdssm_gated_norm, bdssm_residual_norm) against float64 numpy on
the same rounded inputs, element by element.

Bounds, from the arithmetic: float32 products, sums, exp, reciprocal and reciprocal square root
each err by at most a few 2^-24 of their result; a row sum of n terms in float32 by at most
n 2^-24 of the sum of magnitudes (the kernels' trees err far less), which enters the result
halved through the square root; exp(-z) errs by |z| 2^-23. EPS32(n, z) below adds these with room
for ten roundings. A bf16 result adds half a unit in its last place (8 significant bits)."""
import numpy as np
import pytest

from bidirectional_mamba_state_amd import bdssm

pytestmark = pytest.mark.gpu

F32, BF16 = bdssm.F32, bdssm.BF16
EPS = 1e-5


def eps32(n, zmax=0.0):
    return (n / 2 + 2 * zmax + 32) * 2.0**-24


def _t(a, dtype):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()
    return t.bfloat16() if dtype == BF16 else t


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _check(got, want, scale, dtype, n, zmax=0.0, what=""):
    """|got - want| <= eps32 * scale (+ half a unit in the last place for bf16)."""
    tol = eps32(n, zmax) * scale + 1e-30
    if dtype == BF16:
        tol = tol * 1.01 + half_ulp(np.abs(want) + tol)
    worst = float(np.max(np.abs(got - want) / tol)) if got.size else 0.0
    print(f"[parity] {what}: largest error {worst:.3f} of its bound", flush=True)
    assert np.all(np.isfinite(got)) and worst <= 1.0, what


def half_ulp(v):
    """Half a unit in the last place of a bf16 value of magnitude |v|: 2^(e - 8) in [2^e, 2^(e+1))."""
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0**-126))) - 8)


def _rms(v, n):
    return v / np.sqrt((v * v).sum(-1, keepdims=True) / n + EPS)


SHAPES = [  # rows, width, groups: every lanes-per-row and pieces-per-lane variant, odd widths
    (1, 1, 1), (3, 7, 1), (5, 64, 1), (17, 250, 2), (33, 256, 1), (9, 505, 1), (2, 512, 1), (4, 1001, 1),
    (7, 1024, 2), (3, 2048, 1), (5, 2048, 8), (2, 2049, 1), (3, 4000, 1), (2, 5120, 8), (2, 8191, 1), (2, 16384, 1),
    (1, 32768, 2),
]


@pytest.mark.parametrize("rows,width,groups", SHAPES)
@pytest.mark.parametrize("types", [(F32, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("norm_first", [False, True])
def test_gated_norm(rows, width, groups, types, norm_first):
    import torch
    xt, dt = types
    rng = np.random.default_rng(rows * 31 + width + 7 * groups)
    y = _t(rng.standard_normal((rows, width)) * np.exp(rng.uniform(-3, 3, (rows, 1))), xt)
    zx = _t(3 * rng.standard_normal((rows, 2 * width + 3)), dt)  # the gate is a slice of longer rows
    z = zx[:, width:2 * width]
    w = _t(1 + 0.2 * rng.standard_normal(width), F32)
    out = torch.full((rows, width), float("nan"), dtype=torch.bfloat16 if dt == BF16 else torch.float32, device="cuda")
    nd = bdssm.norm_dims(rows, width, dt, groups=groups, eps=EPS, x_dtype=xt)
    print(f"[case] gated {rows}x{width} groups {groups} types {types} first {norm_first}", flush=True)
    bdssm.gated_norm(nd, y, z, w, out, norm_first=norm_first)
    torch.cuda.synchronize()
    yv, zv, wv, n = _np(y), _np(z), _np(w), width // groups
    g = zv / (1 + np.exp(-zv))
    part = lambda v: v.reshape(rows, groups, n)  # noqa: E731
    want = _rms(part(yv), n).reshape(rows, width) * wv * g if norm_first else \
        _rms(part(yv * g), n).reshape(rows, width) * wv
    _check(_np(out), want, np.abs(want), dt, n, float(np.abs(zv).max()), "out")
    again = torch.empty_like(out)
    bdssm.gated_norm(nd, y, z, w, again, norm_first=norm_first)
    assert torch.equal(out, again)


def test_gated_norm_in_place_no_weight_and_extreme_gates():
    import torch
    rows, width = 6, 640
    rng = np.random.default_rng(3)
    y = _t(rng.standard_normal((rows, width)), F32)
    zv = rng.standard_normal((rows, width))
    zv[0, :5] = [-3e38, -1000.0, -100.0, 100.0, 1000.0]  # exp(-z) overflows, or vanishes
    zv[1] = 0.0                                             # a row of zeros after the gate
    z = _t(zv, F32)
    nd = bdssm.norm_dims(rows, width, F32, eps=EPS)
    keep = y.clone()
    bdssm.gated_norm(nd, y, z, None, y)
    torch.cuda.synchronize()
    zd = _np(z)
    with np.errstate(over="ignore"):
        g = zd / (1 + np.exp(-zd))
    want = _rms(_np(keep) * g, width)
    _check(_np(y), want, np.abs(want), F32, width, 100.0, "in place")
    assert torch.count_nonzero(y[1]) == 0


@pytest.mark.parametrize("rows,width", [(1, 1), (6, 7), (10, 64), (4, 250), (64, 505), (8, 1001), (6, 1024), (4, 2560),
                                        (2, 4099), (2, 10000), (3, 16384)])
@pytest.mark.parametrize("types", [(F32, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("layer,post,mod", [(False, True, True), (True, True, True), (True, False, False),
                                            (False, False, True)])
def test_residual_norm(rows, width, types, layer, post, mod):
    import torch
    xt, dt = types
    rps = 2 if rows % 2 == 0 else rows
    streams = -(-rows // rps)
    rng = np.random.default_rng(rows * 17 + width + 5 * layer + post)
    x = _t(rng.standard_normal((rows, width)) + 0.5, xt)
    o = _t(rng.standard_normal((rows, width)) * 3 - 1, dt)
    pw = _t(1 + 0.2 * rng.standard_normal(width), F32) if post else None
    w = _t(1 + 0.2 * rng.standard_normal(width), F32)
    m = _t(rng.standard_normal((streams, 3 * width + 1)), dt)
    part = (lambda i: m[:, i * width:(i + 1) * width]) if mod else (lambda i: None)
    td = torch.bfloat16 if dt == BF16 else torch.float32
    x_out = torch.empty_like(x)
    u = torch.full((rows, width), float("nan"), dtype=td, device="cuda")
    nd = bdssm.norm_dims(rows, width, dt, eps=EPS, rows_per_stream=rps, x_dtype=xt,
                         kind=bdssm.NORM_LAYER if layer else bdssm.NORM_RMS)
    print(f"[case] residual {rows}x{width} types {types} layer {layer} post {post} mod {mod}", flush=True)
    bdssm.residual_norm(nd, x, o, w, x_out, u, post_w=pw, gate=part(0), gain=part(1), shift=part(2), res_scale=0.75)
    torch.cuda.synchronize()

    def norm(v):  # and the scale of its rounding errors: the mean is subtracted from both
        mu = v.mean(-1, keepdims=True) if layer else 0.0
        r = 1 / np.sqrt(((v - mu) ** 2).mean(-1, keepdims=True) + EPS)
        return (v - mu) * r, (np.abs(v) + np.abs(v).mean(-1, keepdims=True) * layer) * r, r

    rows_of = np.arange(rows) // rps
    xv, t = _np(x), _np(o)
    ts = np.abs(t)
    if post:
        t, ts, _ = norm(t)
        t, ts = t * _np(pw), ts * np.abs(_np(pw))
    if mod:
        t, ts = t * _np(part(0))[rows_of], ts * np.abs(_np(part(0))[rows_of])
    r = xv + 0.75 * t
    rs = np.abs(xv) + 0.75 * ts
    _check(_np(x_out), r, rs, xt, width, what="x_out")
    un, us, inv = norm(r)
    # errors of r (relative to rs) pass through the norm, and through its mean square
    us = us + rs * inv + np.abs(un) * (np.abs(un) * rs * inv).mean(-1, keepdims=True) + rs.mean(-1, keepdims=True) * inv
    un, us = un * _np(w), us * np.abs(_np(w))
    if mod:
        gain, shift = _np(part(1))[rows_of], _np(part(2))[rows_of]
        un, us = un * gain + shift, us * np.abs(gain) + np.abs(shift)
    _check(_np(u), un, 2 * us, dt, width, what="u")


def test_residual_norm_parts():
    """Every output and input that may be left out; x updated in place."""
    import torch
    rows, width = 5, 300
    rng = np.random.default_rng(9)
    x, o, w = _t(rng.standard_normal((rows, width)), F32), _t(rng.standard_normal((rows, width)), F32), \
        _t(rng.standard_normal(width), F32)
    nd = bdssm.norm_dims(rows, width, F32, eps=EPS)
    u, xo = torch.empty_like(x), torch.empty_like(x)
    bdssm.residual_norm(nd, x, None, w, None, u)                 # a plain norm
    want = _rms(_np(x), width) * _np(w)
    _check(_np(u), want, np.abs(want), F32, width, what="norm alone")
    bdssm.residual_norm(nd, x, o, None, xo, None, res_scale=2.0)  # an addition alone
    _check(_np(xo), _np(x) + 2 * _np(o), np.abs(_np(x)) + 2 * np.abs(_np(o)), F32, width, what="sum alone")
    u2, x2 = torch.empty_like(x), x.clone()
    bdssm.residual_norm(nd, x2, o, w, x2, u2, res_scale=2.0)      # in place
    u3 = torch.empty_like(x)
    bdssm.residual_norm(nd, x, o, w, xo, u3, res_scale=2.0)
    assert torch.equal(x2, xo) and torch.equal(u2, u3)
    empty = bdssm.norm_dims(0, width, F32, eps=EPS)
    bdssm.residual_norm(empty, x[:0], None, w, None, u[:0])


def test_norms_on_another_stream():
    import torch
    rows, width = 64, 2048
    rng = np.random.default_rng(5)
    y, z = _t(rng.standard_normal((rows, width)), BF16), _t(rng.standard_normal((rows, width)), BF16)
    nd = bdssm.norm_dims(rows, width, BF16, eps=EPS)
    a, b = torch.empty_like(y), torch.empty_like(y)
    bdssm.gated_norm(nd, y, z, None, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    bdssm.gated_norm(nd, y, z, None, b, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
