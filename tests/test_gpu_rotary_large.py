"""Rotary positions of more rows than the GPU's L2s hold (32 MB), which other kernels store: on both
sides of that size, against the definition (some rows of each stream; bounds as in test_gpu_rotary.py)
and, to the last bit, against the same rows in a call a stream."""
import numpy as np
import pytest

from bidirectional_mamba_state_amd import bdssm
from test_gpu_attn import BF16, F32, _case, _np
from test_gpu_rotary import Rows, frequencies, near, turned

pytestmark = pytest.mark.gpu

H, KV, D, PAGE = 4, 2, 64, 64
LAYOUTS = [(64, False), (32, False), (48, True)]


def rows(dtype, above):
    """Streams of a length each, one of none, whose turned rows together end a row below 32 MB or above."""
    n = (32 << 20) // ((H + KV) * D * (2 if dtype == BF16 else 4)) + above
    counts = [n // 3, 0, n // 4, 1]
    counts.append(n - sum(counts))
    return Rows([5, 100, 0, 63, 200], counts, H=H, KV=KV, D=D, dtype=dtype, page=PAGE)


def definition(r, got, raw, dim, interleaved, what):
    g = np.random.default_rng(len(what))
    at = np.unique(np.concatenate([g.integers(0, r.n, 1500), [0, r.n - 1], np.cumsum(r.counts)[:-1] - 1]))
    near(got[at], *turned(_np(raw[at]), r.pos[at], frequencies(dim), interleaved, 1.0), r.dtype, what)


def by_stream(r, f):
    """f(stream, its dims, its rows) for every stream that has some."""
    a = 0
    for b, n in enumerate(r.counts):
        if n:
            f(b, bdssm.attn_dims(1, H, KV, D, r.dtype, PAGE), slice(a, a + n))
        a += n


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,interleaved", LAYOUTS)
@pytest.mark.parametrize("above", [0, 1])
def test_step(dtype, dim, interleaved, above):
    import torch
    _case(f"large rotary dim {dim} dtype {dtype} above {above}")
    r = rows(dtype, above)
    rot = bdssm.Rotary(bdssm.rotary_turns(dim), interleaved)
    qo, ko, q2, k2 = (torch.full((r.n, h, D), 9.0, dtype=r.td, device="cuda") for h in (H, KV, H, KV))
    bdssm.rotary_step(r.ad, r.T, rot, r.q, r.k, qo, ko, lens=r.lens_d, starts=r.starts)
    by_stream(r, lambda b, ad, s: bdssm.rotary_step(ad, r.counts[b], rot, r.q[s], r.k[s], q2[s], k2[s], lens=r.lens_d[b:b + 1]))
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    definition(r, qo, r.q, dim, interleaved, "q")
    definition(r, ko, r.k, dim, interleaved, "k")
    # in place, on slices of the projection: what lies beside them stays
    before = r.qkv.clone()
    bdssm.rotary_step(r.ad, r.T, rot, r.q, r.k, r.q, r.k, lens=r.lens_d, starts=r.starts)
    assert torch.equal(r.q, qo) and torch.equal(r.k, ko)
    assert torch.equal(r.qkv[:, (H + KV) * D:], before[:, (H + KV) * D:])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,interleaved", LAYOUTS)
@pytest.mark.parametrize("above", [0, 1])
@pytest.mark.parametrize("k_out", [False, True])
def test_append(dtype, dim, interleaved, above, k_out):
    """Tokens of pages that are not held, and past the table, are dropped; rows of no stream stay."""
    import torch
    _case(f"large rotary append dim {dim} dtype {dtype} above {above} k_out {k_out}")
    r = rows(dtype, above)
    r.table = r.table[:, :r.table.shape[1] - 2].contiguous()  # the longest stream has no room for its last
    r.table[0, 3], r.table[2, 1] = -1, 1 << 20
    rot = bdssm.Rotary(bdssm.rotary_turns(dim), interleaved)
    qo, ko, q2, k2 = (torch.full((r.n, h, D), 9.0, dtype=r.td, device="cuda") for h in (H, KV, H, KV))
    kp, vp = r.kp.clone(), r.vp.clone()
    lens, lens2 = torch.zeros_like(r.lens_d), r.lens_d.clone()
    cache = bdssm.KvCache(r.ad, kp, vp, r.table, r.lens_d, max(r.lens))
    bdssm.rotary_append(r.ad, r.T, rot, r.q, r.k, r.v, cache, qo, ko if k_out else None, lens, starts=r.starts)

    def one(b, ad, s):
        cache = bdssm.KvCache(ad, r.kp, r.vp, r.table[b:b + 1], r.lens_d[b:b + 1], r.lens[b])
        bdssm.rotary_append(ad, r.counts[b], rot, r.q[s], r.k[s], r.v[s], cache, q2[s], k2[s], lens2[b:b + 1])

    by_stream(r, one)
    held = r.table.shape[1] * PAGE
    assert lens.tolist() == lens2.tolist() == [min(L + n, held) for L, n in zip(r.lens, r.counts)]
    assert torch.equal(qo, q2) and (torch.equal(ko, k2) if k_out else (ko == 9.0).all())
    assert torch.equal(kp, r.kp) and torch.equal(vp, r.vp)
    definition(r, qo, r.q, dim, interleaved, "q")
    definition(r, k2, r.k, dim, interleaved, "k")
    # the pages of every stream hold its keys and values, all but the dropped ones, and no other slot changed
    want_k, want_v = torch.full_like(kp, 3.0), torch.full_like(vp, 4.0)
    a = 0
    for b, (L, n) in enumerate(zip(r.lens, r.counts)):
        j = torch.arange(L, min(L + n, held), device="cuda")
        if len(j):
            page = r.table[b].long()[j // PAGE]
            ok = (page >= 0) & (page < kp.shape[0])
            want_k[page[ok], :, j[ok] % PAGE] = k2[a:a + len(j)][ok]
            want_v[page[ok], :, j[ok] % PAGE] = r.v[a:a + len(j)][ok]
        a += n
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
