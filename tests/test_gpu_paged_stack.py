"""Rotary positions, shaped scores and page upkeep as a decoding loop uses them together: against a
dense definition in float64, and in the example stack (examples/hybrid_stack.py)."""
import numpy as np
import pytest

from bidirectional_mamba_state_amd import bdssm
from test_gpu_attn import BF16, F32, _case, _np, half_ulp
from test_gpu_hybrid import _module, _rel, _stack
from test_gpu_rotary import frequencies, turned

pytestmark = pytest.mark.gpu


class Loop:
    """An attention layer's decoding loop over a managed cache, and beside it every stream's tokens as
    they were given, in float64."""

    def __init__(self, dtype, H=4, KV=2, D=64, page=16, batch=4, per=24, P=60, window=0, sinks=0, cap=0.0, bias=True, seed=0):
        import torch
        self.__dict__.update(dtype=dtype, H=H, KV=KV, D=D, page=page, batch=batch, per=per, P=P, window=window, sinks=sinks,
                             cap=cap)
        self.td = torch.bfloat16 if dtype == BF16 else torch.float32
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.lens, self.lens2, self.uses = z(batch, per) - 1, z(batch), z(batch), z(P)
        self.lacking, self.copies, self.table2 = z(1), z(batch, 2), z(batch, per)
        self.moves = z(P // 2, 2)
        self.kp, self.vp = (torch.full((P, KV, page, D), float("nan"), dtype=self.td, device="cuda") for _ in range(2))
        self.ad = bdssm.attn_dims(batch, H, KV, D, dtype, page)
        self.pd = bdssm.page_dims(batch, page, P, per)
        self.ws = torch.empty(bdssm.pages_workspace(self.pd), dtype=torch.uint8, device="cuda")
        self.rot = bdssm.Rotary(bdssm.rotary_turns(D))
        self.slopes = [2.0 ** -(h + 1) for h in range(H)] if bias else [0.0] * H
        s = torch.tensor(self.slopes, device="cuda") if bias else None
        self.scores = bdssm.AttnScores(cap=cap, slopes=s)
        self.mask = bdssm.attn_mask(D ** -0.5, 1, window, sinks)
        self.cache = bdssm.KvCache(self.ad, self.kp, self.vp, self.table, self.lens, per * page)
        self.books = bdssm.Pages(self.pd, self.table, self.lens, self.uses)
        self.k = [np.zeros((0, KV, D)) for _ in range(batch)]  # turned, rounded: what the cache should hold
        self.v = [np.zeros((0, KV, D)) for _ in range(batch)]

    def block(self, counts):
        """New tokens of every stream: pages taken, keys turned into them, attention before the lengths
        move on. Checks every row."""
        import torch
        n, T = sum(counts), max(counts)
        starts = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        H, KV, D = self.H, self.KV, self.D
        qkv = torch.randn((n, (H + 2 * KV) * D), generator=self.g, device="cuda").to(self.td)
        q, k, v = (qkv[:, a * D:(a + h) * D].view(n, h, D) for a, h in ((0, H), (H, KV), (H + KV, KV)))
        raw_q, raw_k = _np(q), _np(k)
        bdssm.pages_advance(self.pd, self.books, T, self.table, self.uses, self.lacking, self.ws, self.window, self.sinks,
                            starts)
        assert int(self.lacking) == 0
        bdssm.rotary_append(self.ad, T, self.rot, q, k, v, self.cache, q, k, self.lens2, starts=starts)
        out = torch.full((n, H, D), float("nan"), dtype=self.td, device="cuda")
        need = bdssm.attn_step_ex_workspace(self.ad, T, self.per * self.page, self.mask, self.scores)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        bdssm.attn_step_ex(self.ad, T, q, k, v, self.cache, self.mask, self.scores, out, ws, starts=starts)
        pos = np.concatenate([np.arange(len(self.k[b]), len(self.k[b]) + c) for b, c in enumerate(counts)])
        f = frequencies(D)
        for got, raw in ((q, raw_q), (k, raw_k)):
            want, tol = turned(raw, pos, f, False, 1.0)
            if self.dtype == BF16:
                tol = tol + half_ulp(np.abs(want) + tol)
            assert (np.abs(_np(got) - want) <= tol).all()
        at = 0
        for b, c in enumerate(counts):
            self.k[b] = np.concatenate([self.k[b], _np(k[at:at + c])])
            self.v[b] = np.concatenate([self.v[b], _np(v[at:at + c])])
            self.check(b, _np(q[at:at + c]), _np(out[at:at + c]))
            at += c
        self.lens.copy_(self.lens2)

    def check(self, b, q, out):
        e, K, V, G = 2.0**-24, self.k[b], self.v[b], self.H // self.KV
        for i in range(len(q)):
            p = len(K) - len(q) + i
            j = np.arange(p + 1)
            j = j[(p - j < self.window) | (j < self.sinks)] if self.window else j
            for h in range(self.H):
                Kh, Vh = K[j, h // G], V[j, h // G]
                s = Kh @ q[i, h] * self.D ** -0.5
                S = (np.abs(Kh) @ np.abs(q[i, h])).max() * self.D ** -0.5
                s = (self.cap * np.tanh(s / self.cap) if self.cap else s) - self.slopes[h] * (p - j)
                w = np.exp(s - s.max())
                w /= w.sum()
                o, W = w @ Vh, w @ np.abs(Vh)
                E = e * ((self.D + 40) * S + 8 * self.slopes[h] * (p - j))  # as in test_gpu_attn_scored.py
                t = (w * E) @ np.abs(Vh) + W * ((w @ E) + e * 2 * (len(j) + 16))
                if self.dtype == BF16:
                    t = 1.01 * (t + 2.0**-8 * W)
                    t = t + half_ulp(np.abs(o) + t)
                assert (np.abs(out[i, h] - o) <= t).all(), (b, i, h)

    def fork(self, parents):
        import torch
        p = torch.tensor(parents, dtype=torch.int32, device="cuda")
        bdssm.pages_fork(self.pd, self.books, p, self.table2, self.lens2, self.uses, self.copies, self.lacking, self.ws)
        bdssm.pages_copy(self.ad, self.cache, self.copies)
        self.table.copy_(self.table2)
        self.lens.copy_(self.lens2)
        empty = np.zeros((0, self.KV, self.D))
        self.k, self.v = ([x[p] if 0 <= p < self.batch else empty for p in parents] for x in (self.k, self.v))

    def compact(self):
        live = self.lacking.clone()
        bdssm.pages_compact(self.pd, self.books, self.table, self.uses, self.moves, live, self.ws)
        bdssm.pages_copy(self.ad, self.cache, self.moves)
        n = int(live)
        assert (self.uses[:n] > 0).all() and not self.uses[n:].any()
        self.kp[n:] = float("nan")  # nothing is left there
        self.vp[n:] = float("nan")
        return n


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks,cap", [(0, 0, 0.0), (0, 0, 8.0), (40, 3, 8.0)])
def test_a_decoding_loop(dtype, window, sinks, cap):
    """Prompts, blocks, forks into several continuations, ended streams, compactions: at every step
    each stream attends to its own tokens."""
    _case(f"loop dtype {dtype} window {window} cap {cap}")
    s = Loop(dtype, window=window, sinks=sinks, cap=cap)
    s.block([50, 3, 16, 0])
    s.block([1, 1, 1, 1])
    s.fork([0, 0, 2, 0])
    s.block([20, 7, 16, 33])
    n = s.compact()
    s.block([5, 5, 5, 5])
    s.fork([3, -1, 1, 3])
    s.block([2, 30, 1, 2])
    s.fork([0, 1, 2, 3])
    assert s.compact() <= s.P and n > 0
    for _ in range(3):
        s.block([17, 1, 16, 9])


def test_the_loops_block_in_a_graph():
    """A block's upkeep, rotary append and attention recorded once: replays go on from block to block as
    the eager calls do."""
    import torch
    _case("loop in a graph")
    T, n = 8, 32
    outs = []
    for graphed in (False, True):
        s = Loop(BF16, window=30, sinks=2, cap=5.0, seed=3)
        s.block([40, 5, 16, 1])
        g = torch.Generator(device="cuda")
        g.manual_seed(9)
        x = torch.zeros((n, 8 * 64), dtype=torch.bfloat16, device="cuda")
        q, k, v = (x[:, a * 64:(a + h) * 64].view(n, h, 64) for a, h in ((0, 4), (4, 2), (6, 2)))
        out = torch.zeros((n, 4, 64), dtype=torch.bfloat16, device="cuda")
        need = bdssm.attn_step_ex_workspace(s.ad, T, s.per * s.page, s.mask, s.scores)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")

        def block():
            bdssm.pages_advance(s.pd, s.books, T, s.table, s.uses, s.lacking, s.ws, s.window, s.sinks)
            bdssm.rotary_append(s.ad, T, s.rot, q, k, v, s.cache, q, k, s.lens2)
            bdssm.attn_step_ex(s.ad, T, q, k, v, s.cache, s.mask, s.scores, out, ws)
            s.lens.copy_(s.lens2)

        def fill():
            x.copy_(torch.randn(x.shape, generator=g, device="cuda").bfloat16())

        side = torch.cuda.Stream()
        fill()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            block()
        torch.cuda.current_stream().wait_stream(side)
        got = [out.clone()]
        run = block
        if graphed:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                block()
            run = graph.replay
        for _ in range(6):
            fill()
            run()
            torch.cuda.synchronize()
            got.append(out.clone())
        outs.append((got, s.table.clone(), s.uses.clone(), s.lens.clone()))
    a, b = outs
    assert all(torch.equal(x, y) for x, y in zip(a[0], b[0]))
    assert all(torch.equal(x, y) for x, y in zip(a[1:], b[1:]))
    assert torch.isfinite(torch.stack(a[0])).all()


OPTIONS = dict(rotary=True, cap=20.0, bias=True, managed=True)


@pytest.mark.parametrize("window", [0, 40])
def test_the_stacks_prompt_at_once_equals_commits(window):
    """As the plain stack's (tests/test_gpu_hybrid.py), with every option on."""
    import torch
    m = _module()
    one, many = (_stack(m, window=window, sinks=4 if window else 0, **OPTIONS) for _ in range(2))
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn((2, 96, 256), generator=g, device="cuda")
    one.prefill(x.reshape(-1, 256).clone(), 96)
    for i in range(0, 96, 32):
        many.commit(x[:, i:i + 32].reshape(-1, 256).clone())
    assert one.lens[0].tolist() == many.lens[0].tolist() == [96, 96]
    noisy = torch.randn((64, 256), generator=g, device="cuda")
    t = torch.full((2,), 0.5, device="cuda")
    ya, yb = one.denoise(noisy.clone(), t), many.denoise(noisy.clone(), t)
    assert torch.isfinite(ya).all() and _rel(ya, yb) < 0.05


def test_managed_pages_and_compaction_change_nothing():
    """The same stack with pages held from the start, managed, and managed and compacted: the same
    bits."""
    import torch
    m = _module()
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    x = torch.randn((3, 64, 256), generator=g, device="cuda")
    noisy, t = torch.randn((64, 256), generator=g, device="cuda"), torch.full((2,), 0.4, device="cuda")
    outs = []
    for managed, compact in ((False, False), (True, False), (True, True)):
        s = _stack(m, rotary=True, cap=20.0, managed=managed, window=48, sinks=4)
        for block in x:
            s.commit(block.clone())
            if compact:
                live = int(s.compact())
                assert live == int((s.uses > 0).sum())
        outs.append(s.denoise(noisy.clone(), t))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_forked_streams_continue_their_parent():
    """Two streams forked from one decode as that one does; its pages are shared, and the partly
    filled one is not."""
    import torch
    m = _module()
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    prompt, nxt = torch.randn((2, 96, 256), generator=g, device="cuda"), torch.randn((32, 256), generator=g, device="cuda")
    s = _stack(m, **OPTIONS)
    s.prefill(prompt.reshape(-1, 256).clone(), 96)
    before = int((s.uses > 0).sum())
    s.fork(torch.tensor([1, 1], dtype=torch.int32, device="cuda"))
    assert s.uses.max().item() == 2 and int((s.uses > 0).sum()) == before - 1  # a whole page shared, a page each
    both = torch.cat([nxt, nxt])
    t = torch.full((2,), 0.5, device="cuda")
    y = s.denoise(both.clone(), t).view(2, 32, 256)
    assert torch.equal(y[0], y[1])
    s.commit(both.clone())
    other = torch.randn((64, 256), generator=g, device="cuda")
    s.commit(other.clone())  # the two part ways
    y = s.denoise(both.clone(), t).view(2, 32, 256)
    ref = _stack(m, **OPTIONS)
    ref.prefill(prompt[1].repeat(2, 1, 1).reshape(-1, 256).clone(), 96)
    ref.commit(both.clone())
    ref.commit(other.clone())
    assert torch.equal(ref.denoise(both.clone(), t).view(2, 32, 256), y)
    assert not torch.equal(y[0], y[1])


@pytest.mark.parametrize("argv", [[], ["--rotary", "--cap", "30", "--samples", "3"], ["--bias", "--window", "64"]])
def test_the_example_runs(argv, capsys, monkeypatch):
    import sys
    m = _module()
    monkeypatch.setattr(sys, "argv", ["hybrid_stack.py", "--tiny", "--steps", "2", *argv])
    m.main()
    assert "block 1" in capsys.readouterr().out
