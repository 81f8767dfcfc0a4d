"""Launch plans of bdssm_attn_step on the GPU: one workspace for many lengths."""
import numpy as np
import pytest

from bidirectional_mamba_state_amd import bdssm
from test_gpu_attn import Case, _case, _np, half_ulp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,KV,lens", [(40, 8, (5600, 6016, 7296, 7777, 8064)), (24, 4, (7616, 8000, 8064))])
def test_the_longest_caches_workspace_serves_shorter_ones(H, KV, lens):
    """A block of 32 on 8,192 cached tokens takes fewer ranges than on some shorter caches."""
    import torch
    longest = 8192
    c = Case([longest], [32], H=H, KV=KV, page=32)
    ws = torch.full((bdssm.attn_step_workspace(c.ad, 32, longest, c.mask),), 255, dtype=torch.uint8, device="cuda")
    for n in (*lens, 1000, 1, longest):
        _case(f"{H} heads over {KV}, {n} of {longest} tokens")
        c.lens, c.max_len = [n], n
        c.lens_d.fill_(n)
        c.cache.max_len = n
        out = torch.full_like(c.q, float("nan"))
        bdssm.attn_step(c.ad, 32, c.q, c.k, c.v, c.cache, c.mask, out, ws)
        torch.cuda.synchronize()
        if n in (lens[0], 1000):
            want, tol = c.want()
            assert np.all(np.abs(_np(out) - want) <= tol)
        assert torch.equal(out, c.run())  # with a workspace of its own length


@pytest.mark.parametrize("dtype", [bdssm.BF16, bdssm.F32])
@pytest.mark.parametrize("block", [0, 250])
def test_window_over_a_chunk_that_looks_ahead(dtype, block):
    """Queries that see few keys back and many ahead, their keys split over workgroups."""
    _case(f"window without order, {dtype} {block}")
    c = Case([90], [700], H=2, KV=1, dtype=dtype, block=block, window=37, sinks=5, page=32)
    assert bdssm.attn_step_workspace(c.ad, 700, 90, c.mask) > 0
    c.check("window without order")


@pytest.mark.parametrize("D,block", [(64, 0), (128, 32)])
def test_few_units_of_many_row_tiles(D, block):
    """The launch of a prompt, in small: 33 (stream, KV head) pairs of nine row tiles, dealt to the
    XCDs in two parts each, tile by tile. All rows against float64, within the bounds of
    test_gpu_attn.py's docstring."""
    _case(f"many row tiles {D} {block}")
    b, T, G, e = 33, 33, 64, 2.0**-24
    lens = [500 - 7 * i for i in range(b)]
    c = Case(lens, [T] * b, H=G, KV=1, D=D, block=block, page=64)
    got = _np(c.run()).reshape(b, T, G, D)
    q, k, v = (_np(t).reshape(b, T, -1, D) for t in (c.q, c.k, c.v))
    kp, vp, table = _np(c.kp)[:, 0], _np(c.vp)[:, 0], c.table.cpu().numpy()
    for i, n in enumerate(lens):
        K = np.concatenate([kp[table[i]].reshape(-1, D)[:n], k[i, :, 0]])
        V = np.concatenate([vp[table[i]].reshape(-1, D)[:n], v[i, :, 0]])
        at, p = np.arange(n + T), n + np.arange(T)
        see = np.ones((T, n + T), bool) if block == 0 else at[None] // block <= p[:, None] // block
        see = see[:, None, :]
        s = np.where(see, c.scale * (q[i] @ K.T), -np.inf)
        w = np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        want, W = w @ V, w @ np.abs(V)
        S = np.where(see, c.scale * (np.abs(q[i]) @ np.abs(K).T), 0.0).max(-1, keepdims=True)
        tol = W * e * (4 * (D + 8) * S + 8 * S + 2 * (n + T + 16))
        tol = 1.01 * (tol + 2.0**-8 * W)
        tol = tol + half_ulp(np.abs(want) + tol)
        assert np.all(np.abs(got[i] - want) <= tol), i
