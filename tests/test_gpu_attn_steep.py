"""bdssm_attn_step_ex with slopes so steep that a row's nearest key takes all of its weight, up to the
end of float32's range, and with scores near the end of what the call holds.

Bounds: the one weight that is left is the sum too, so that a result is the value times weight /
weight: the product, the inverse and their product round three times in float32 (3 x 2^-24 of it),
which bf16's rounding, the value being bf16, takes away."""
import numpy as np
import pytest

from bidirectional_mamba_state_amd import bdssm
from test_gpu_attn import BF16, F32, _case, _np
from test_gpu_attn_scored import Scored

pytestmark = pytest.mark.gpu

SLOPES = [2.0**29, 2.0**64, 1.5 * 2.0**97, 3e38]
SHAPES = [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)]


def only(c, at, what):
    """Every row is the value at position at[row] (of its stream, which is the first)."""
    got = _np(c.run())
    kp, v, table = _np(c.vp), _np(c.v), c.table.cpu().numpy()
    L = c.lens[0]
    G = c.H // c.KV
    for i, j in enumerate(at):
        want = kp[table[0, j // c.page], :, j % c.page] if j < L else v[j - L]
        err = np.abs(got[i] - np.repeat(want, G, axis=0))
        bound = 0.0 if c.dtype == BF16 else 3 * 2.0**-24
        assert (err <= bound * np.abs(np.repeat(want, G, axis=0))).all(), (what, i, j)


def with_scale(c, scale):
    """The same scores from another scale, up to its power of two."""
    import math
    c.q.mul_(2.0 ** -round(math.log2(scale / c.scale)))
    c.scale = scale
    c.mask = bdssm.attn_mask(scale, c.block, c.window, c.sinks)
    return c


@pytest.mark.parametrize("dtype,D", SHAPES)
@pytest.mark.parametrize("cap", [0.0, 30.0, 400.0])
@pytest.mark.parametrize("scale", [None, 2.0**-64, 2.0**64])
def test_the_nearest_key_is_left(dtype, D, cap, scale):
    """At any place among the keys of a tile, of the cache and of the chunk."""
    _case(f"steep D {D} dtype {dtype} cap {cap} scale {scale}")
    for n, H in ((100, 4), (7, 4)):
        make = lambda **kw: with_scale(Scored([100], [n], H=H, D=D, dtype=dtype, cap=cap, slopes=SLOPES, **kw),  # noqa: E731
                                       scale or D**-0.5)
        only(make(own_keys=False), [99] * n, "the cache's last")
        only(make(own_keys=False, last=[i + 1 for i in range(n)]), list(range(n)), "the range's last")
        only(make(block=1), [100 + i for i in range(n)], "its own")
        only(make(window=9, sinks=3), [100 + i for i in range(n)], "its own, in a window")
        only(make(window=9, sinks=40, own_keys=False, last=[60] * n), [39] * n, "the last sink")
        only(make(first=[100 + n - 1] * n), [100 + n - 1] * n, "the chunk's last")


@pytest.mark.parametrize("dtype,D", SHAPES)
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_scores_near_the_end(dtype, D, cap):
    """A slope below zero favours the farthest key, here with scores of 2^19 to 2^29."""
    _case(f"rising D {D} dtype {dtype} cap {cap}")
    c = Scored([100], [40], D=D, dtype=dtype, cap=cap, block=1, slopes=[-2.0**29 / 139, -2.0**20, -2.0**12, -2.0**22])
    only(c, [0] * 40, "the farthest")


@pytest.mark.parametrize("dtype,D", SHAPES)
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_far_keys_before_the_nearest(dtype, D, cap):
    """Slopes below the limit whose products with the distance pass it (or just do not), over many tiles: the
    tiles of far keys come first, in the cache and in a chunk without order."""
    _case(f"far keys D {D} dtype {dtype} cap {cap}")
    for slopes in ([2.0**26, 2.0**25, 1e7, 1e6], [2.0**26 / 3000, 2.0**26 / 2999, 2.0**15, 1e4]):
        make = lambda lens, n, **kw: Scored([lens], [n], D=D, dtype=dtype, cap=cap, slopes=slopes, **kw)  # noqa: E731
        for n in (2, 70):
            only(make(3000, n, own_keys=False), [2999] * n, "the cache's last")
            only(make(3000, n, own_keys=False, last=[1000 + i for i in range(n)]), [999 + i for i in range(n)], "the range's")
        only(make(70, 600), [70 + i for i in range(600)], "its own")


@pytest.mark.parametrize("dtype,D", SHAPES)
def test_steep_slopes_beside_infinities(dtype, D):
    """The rows that are computed again beside an infinity."""
    _case(f"steep beside infinities D {D} dtype {dtype}")
    for cap in (0.0, 30.0):
        c = Scored([100], [50], D=D, dtype=dtype, cap=cap, block=1, slopes=SLOPES)
        c.v[49] = float("inf")
        got = _np(c.run())
        assert np.isinf(got[49]).all()
        want = np.repeat(_np(c.v)[:49], 2, axis=1)
        assert (np.abs(got[:49] - want) <= 3 * 2.0**-24 * np.abs(want)).all()
