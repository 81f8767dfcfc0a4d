"""Upkeep of a paged cache (bdssm_pages_advance, _fork, _compact, _copy) against plain Python."""
import numpy as np
import pytest

from bidirectional_mamba_state_amd import bdssm
from test_gpu_attn import BF16, F32, _case

pytestmark = pytest.mark.gpu


class Model:
    """Table, lengths and uses as numpy arrays, and what the calls do to them, one entry at a time."""

    def __init__(self, table, lens, uses, page):
        self.table, self.lens, self.uses = (np.array(x, dtype=np.int32) for x in (table, lens, uses))
        self.page = page
        self.P, (self.b, self.per) = len(self.uses), self.table.shape

    def is_page(self, e):
        return 0 <= e < self.P

    def length(self, b):
        return int(min(max(int(self.lens[b]), 0), self.per * self.page))

    def advance(self, counts, window=0, sinks=0):
        uses, free, lacking = np.maximum(self.uses, 0), [p for p in range(self.P) if self.uses[p] <= 0], 0
        out = np.full_like(self.table, -1)
        for b in range(self.b):
            L, page = self.length(b), self.page
            end = min(L + counts[b], self.per * page)
            for i in range(self.per):
                e = int(self.table[b, i])
                seen = window == 0 or i * page < sinks or (i + 1) * page > L - window + 1
                new = i * page >= L
                if self.is_page(e):
                    if i * page < end and (new or seen):
                        out[b, i] = e
                    else:
                        uses[e] -= 1
                elif new and i * page < end:
                    if free:
                        out[b, i] = free.pop(0)
                        uses[out[b, i]] += 1
                    else:
                        lacking += 1
        return out, uses, lacking

    def fork(self, parents):
        uses, free, lacking = np.maximum(self.uses, 0), [p for p in range(self.P) if self.uses[p] <= 0], 0
        out, lens = np.full_like(self.table, -1), np.zeros_like(self.lens)
        copies, seen = np.full((self.b, 2), -1, dtype=np.int32), set()
        for b, p in enumerate(map(int, parents)):
            if not 0 <= p < self.b:
                continue
            L = lens[b] = self.length(p)
            row = [e if self.is_page(e) else -1 for e in map(int, self.table[p])]
            if p in seen:
                whole, part = divmod(L, self.page)
                old = row[whole] if part else -1
                row[whole:] = [-1] * (self.per - whole)
                if old >= 0:
                    if free:
                        row[whole] = free.pop(0)
                        copies[b] = old, row[whole]
                    else:
                        lacking += 1
            seen.add(p)
            out[b] = row
        for old, new in zip(self.table.ravel(), out.ravel()):
            if self.is_page(old):
                uses[old] -= 1
            if new >= 0:
                uses[new] += 1
        return out, lens, uses, copies, lacking

    def compact(self):
        uses = np.maximum(self.uses, 0)
        live = int((uses > 0).sum())
        high, low = [p for p in range(live, self.P) if uses[p] > 0][::-1], [p for p in range(live) if uses[p] == 0]
        copies, to = np.full((self.P // 2, 2), -1, dtype=np.int32), np.arange(self.P)
        for r, (a, b) in enumerate(zip(high, low)):
            copies[r], to[a] = (a, b), b
            uses[b], uses[a] = uses[a], 0
        out = np.array([[to[e] if self.is_page(e) else -1 for e in map(int, row)] for row in self.table],
                       dtype=np.int32).reshape(self.table.shape)
        return out, uses, copies, live


class Device:
    """The same arrays on the device, and the library's calls on them."""

    def __init__(self, m):
        import torch
        d = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.lens, self.uses = d(m.table), d(m.lens), d(m.uses)
        self.table = self.table.view(m.b, m.per)
        self.pd = bdssm.page_dims(m.b, m.page, m.P, m.per)
        self.m, self.pages = m, bdssm.Pages(self.pd, self.table, self.lens, self.uses)
        self.ws = torch.full((bdssm.pages_workspace(self.pd),), 255, dtype=torch.uint8, device="cuda")
        full = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table_out, self.uses_out, self.lens_out = full(m.b, m.per), full(m.P), full(m.b)
        self.copies, self.moves, self.count = full(m.b, 2), full(m.P // 2, 2), full(1)

    def starts(self, counts):
        import torch
        return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")

    def advance(self, counts, window=0, sinks=0, in_place=False, even=False, stream=None):
        t, u = (self.table, self.uses) if in_place else (self.table_out, self.uses_out)
        bdssm.pages_advance(self.pd, self.pages, max(counts, default=0), t, u, self.count, self.ws, window, sinks,
                            None if even else self.starts(counts), stream)
        return t.cpu().numpy(), u.cpu().numpy(), int(self.count)

    def fork(self, parents, in_place=False, stream=None):
        import torch
        u = self.uses if in_place else self.uses_out
        p = torch.tensor(parents, dtype=torch.int32, device="cuda")
        bdssm.pages_fork(self.pd, self.pages, p, self.table_out, self.lens_out, u, self.copies, self.count, self.ws, stream)
        return (self.table_out.cpu().numpy(), self.lens_out.cpu().numpy(), u.cpu().numpy(), self.copies.cpu().numpy(),
                int(self.count))

    def compact(self, in_place=False, stream=None):
        t, u = (self.table, self.uses) if in_place else (self.table_out, self.uses_out)
        bdssm.pages_compact(self.pd, self.pages, t, u, self.moves, self.count, self.ws, stream)
        return t.cpu().numpy(), u.cpu().numpy(), self.moves.cpu().numpy(), int(self.count)


def same(got, want, what):
    assert len(got) == len(want)
    for i, (a, b) in enumerate(zip(got, want)):
        assert np.array_equal(a, b), f"{what}: output {i}\n{a}\n{b}"


def random_cache(g, batch, per, P, page, gaps=0.1, share=0.2):
    """Streams of pages from anywhere in the pool, some shared, some given back, junk numbers among
    the empty entries."""
    table, uses, lens = np.full((batch, per), -1, np.int32), np.zeros(P, np.int32), np.zeros(batch, np.int32)
    free = list(g.permutation(P))
    for b in range(batch):
        lens[b] = g.integers(0, per * page + 1) if g.random() < 0.9 else g.choice([0, page, per * page, page * (per // 2)])
        held = -(-int(lens[b]) // page) + int(g.integers(0, 3))
        for i in range(per):
            if i < held and g.random() > gaps:
                if g.random() < share and b and i < lens[b] // page and 0 <= table[b - 1, i] < P:
                    table[b, i] = table[b - 1, i]
                elif free:
                    table[b, i] = free.pop()
                if 0 <= table[b, i] < P:
                    uses[table[b, i]] += 1
            elif g.random() < 0.3:
                table[b, i] = g.choice([-1, -7, P, P + 5, 2**31 - 1, -2**31])
    uses[uses == 0] = g.choice([0, 0, 0, -3], (uses == 0).sum())
    return Model(table, lens, uses, page)


SHAPES = [(1, 1, 1, 16), (1, 5, 7, 16), (3, 9, 40, 32), (7, 33, 200, 16), (2, 300, 700, 256), (64, 40, 2000, 64),
          (5, 3000, 9000, 16), (300, 3, 4097, 128), (3, 4, 4096, 16), (9, 0, 5, 16), (1024, 16, 16384, 16),
          # more pages, entries or streams than one workgroup takes
          (3, 400, 16385, 16), (4, 16400, 12000, 16), (1025, 4, 4500, 32), (2, 6000, 70000, 64)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_advance(shape, in_place):
    batch, per, P, page = shape
    _case(f"advance {shape} in place {in_place}")
    g = np.random.default_rng(P)
    for trial in range(4):
        m = random_cache(g, batch, per, P, page)
        window, sinks = (0, 0) if trial == 0 else (int(g.integers(1, 4 * page)), int(g.choice([0, 1, 3 * page])))
        even = trial == 1
        counts = [int(g.integers(0, 5 * page))] * batch if even else [int(x) for x in g.integers(0, 5 * page, batch)]
        d = Device(m)
        same(d.advance(counts, window, sinks, in_place, even), m.advance(counts, window, sinks), f"trial {trial}")


@pytest.mark.parametrize("in_place", [False, True])
def test_advance_by_many_pages(in_place):
    """A prompt's pages at once: hundreds of new entries of a stream, some of them held already."""
    _case("many new pages")
    g = np.random.default_rng(2)
    m = random_cache(g, 3, 900, 4000, 16)
    m.lens[:] = [0, 100, 5000]
    same(Device(m).advance([14000, 1040, 5000], 0, 0, in_place), m.advance([14000, 1040, 5000]), "many")
    m = random_cache(g, 2, 90, 400, 16)
    same(Device(m).advance([64 * 16 + 15, 3], 0, 0, in_place), m.advance([64 * 16 + 15, 3]), "at the limit")
    m = random_cache(g, 3, 3000, 9000, 16, gaps=0.3)  # more than a workgroup lists at a time
    m.lens[:] = [0, 700, 0]
    m.table[2] = -1
    m.uses = np.bincount(m.table[(m.table >= 0) & (m.table < m.P)], minlength=m.P).astype(np.int32)
    same(Device(m).advance([40000, 33000, 48000], 0, 0, in_place), m.advance([40000, 33000, 48000]), "thousands")


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_fork(shape, in_place):
    batch, per, P, page = shape
    _case(f"fork {shape} in place {in_place}")
    g = np.random.default_rng(P + 1)
    for trial in range(4):
        m = random_cache(g, batch, per, P, page)
        parents = [list(range(batch)), [batch // 2] * batch, [int(x) for x in g.integers(-1, batch + 1, batch)],
                   [int(x) for x in g.choice([-2**31, 2**31 - 1, 0], batch)]][trial]
        d = Device(m)
        same(d.fork(parents, in_place), m.fork(parents), f"trial {trial}")


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_compact(shape, in_place):
    batch, per, P, page = shape
    _case(f"compact {shape} in place {in_place}")
    g = np.random.default_rng(P + 2)
    for trial in range(4):
        m = random_cache(g, batch, per, P, page, gaps=[0.0, 0.1, 0.6, 1.0][trial])
        d = Device(m)
        same(d.compact(in_place), m.compact(), f"trial {trial}")


def test_full_and_empty_pools():
    _case("full and empty pools")
    for P in (1, 2, 64, 4096, 5000):
        m = Model(np.arange(P)[None], [P * 16], np.ones(P), 16)
        same(Device(m).compact(), m.compact(), "full")
        same(Device(m).advance([16]), m.advance([16]), "full")
        same(Device(m).fork([0]), m.fork([0]), "full")
        m = Model(np.full((2, P), -1), [0, 0], np.zeros(P), 16)
        same(Device(m).compact(), m.compact(), "empty")
        same(Device(m).advance([0, 16 * P]), m.advance([0, 16 * P]), "take all")
    m = Model(np.zeros((0, 4)), [], np.array([1, 0, 2]), 16)
    same(Device(m).advance([]), m.advance([]), "no streams")
    same(Device(m).fork([]), m.fork([]), "no streams")
    same(Device(m).compact(), m.compact(), "no streams")
    m = Model(np.full((2, 3), 5), [7, 9], np.zeros(0), 16)
    same(Device(m).advance([20, 0]), m.advance([20, 0]), "no pages")
    same(Device(m).fork([1, 1]), m.fork([1, 1]), "no pages")
    same(Device(m).compact(), m.compact(), "no pages")


def test_lengths_out_of_range():
    _case("lengths out of range")
    m = Model([[0, 1, 2], [3, -1, -1]], [-5, 1 << 30], [1, 1, 1, 1, 0, 0], 16)
    same(Device(m).advance([40, 5]), m.advance([40, 5]), "advance")
    same(Device(m).fork([1, 0]), m.fork([1, 0]), "fork")


def test_more_streams_than_a_grid_row_of_sums():
    """Thousands of streams, many of one parent: places among the needs of thousands in front."""
    _case("many streams")
    g = np.random.default_rng(9)
    batch = 5000
    m = random_cache(g, batch, 2, 14000, 16)
    parents = [int(x) for x in g.integers(0, 7, batch)]
    same(Device(m).fork(parents), m.fork(parents), "fork")
    counts = [int(x) for x in g.integers(0, 33, batch)]
    same(Device(m).advance(counts), m.advance(counts), "advance")


@pytest.mark.parametrize("dtype,D,KV,page", [(BF16, 64, 1, 16), (BF16, 128, 3, 64), (F32, 64, 2, 32), (F32, 128, 8, 256)])
def test_copy(dtype, D, KV, page):
    """Listed pages are copied whole, in both pools, nothing else changes; entries that name no page
    are left out."""
    import torch
    _case(f"copy dtype {dtype} D {D} KV {KV} page {page}")
    P = 37
    ad = bdssm.attn_dims(1, KV, KV, D, dtype, page)
    td = torch.bfloat16 if dtype == BF16 else torch.float32
    k, v = (torch.randn((P, KV, page, D), device="cuda").to(td) for _ in range(2))
    cache = bdssm.KvCache(ad, k, v, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                          torch.zeros(1, dtype=torch.int32, device="cuda"), 0)
    pairs = [(3, 4), (-1, -1), (36, 0), (5, 5), (3, 9), (P, 1), (2, P + 8), (-2**31, 2**31 - 1), (10, 36 - 1), (7, -1)]
    want = [x.clone() for x in (k, v)]
    for a, b in pairs:
        if 0 <= a < P and 0 <= b < P and a != b:
            for w, x in zip(want, (k, v)):
                w[b] = x[a]
    bdssm.pages_copy(ad, cache, torch.tensor(pairs, dtype=torch.int32, device="cuda"))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    none = torch.full((30000, 2), -1, dtype=torch.int32, device="cuda")
    none[29999, 0], none[29999, 1] = 1, 30
    want[0][30], want[1][30] = k[1], v[1]
    bdssm.pages_copy(ad, cache, none)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_a_pool_past_2_to_the_32_bytes():
    """Pages whose offset in the pool passes 32 bits."""
    import torch
    _case("large pool")
    KV, page, D = 8, 256, 128
    P = 9000  # 4.7 GB a pool
    ad = bdssm.attn_dims(1, KV, KV, D, BF16, page)
    k = torch.zeros((P, KV, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[P - 1], v[P - 2] = 3.0, 5.0
    cache = bdssm.KvCache(ad, k, v, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                          torch.zeros(1, dtype=torch.int32, device="cuda"), 0)
    bdssm.pages_copy(ad, cache, torch.tensor([[P - 1, 1], [P - 2, P - 5]], dtype=torch.int32, device="cuda"))
    assert (k[1] == 3).all() and (v[P - 5] == 5).all() and not v[1].any() and not k[P - 5].any()
    assert not k[2:P - 1].any() and not v[:P - 5].any()


def test_replays_of_a_graph_go_on():
    """A block's upkeep recorded once and replayed: in place, the streams advance from replay to
    replay as in plain Python; on another stream too."""
    import torch
    _case("graph")
    g = np.random.default_rng(4)
    page, per = 16, 60
    m = Model(np.full((6, per), -1), np.zeros(6), np.zeros(150), page)
    d = Device(m)
    counts = torch.tensor([20, 3, 16, 1, 33, 8], dtype=torch.int32, device="cuda")
    starts = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cumsum(counts, 0).to(torch.int32)])

    def block():
        bdssm.pages_advance(d.pd, d.pages, 33, d.table, d.uses, d.count, d.ws, 64, 4, starts)
        d.lens.add_(counts)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    c = counts.tolist()
    for replay in range(12):
        table, uses, lacking = m.advance(c, 64, 4)
        m.table, m.uses = table, uses
        m.lens = m.lens + np.array(c, np.int32)
        if replay:
            graph.replay()
            torch.cuda.synchronize()
        assert np.array_equal(d.table.cpu().numpy(), table), replay
        assert np.array_equal(d.uses.cpu().numpy(), uses), replay
        assert int(d.count) == lacking
        g.random()


def test_a_long_run_of_calls_keeps_the_books():
    """Hundreds of advances, forks, ends and compactions: the uses stay the entries that name a page,
    no page has two writers, and every call is as in plain Python."""
    _case("long run")
    g = np.random.default_rng(11)
    batch, per, P, page = 9, 20, 120, 16
    m = Model(np.full((batch, per), -1), np.zeros(batch), np.zeros(P), page)
    for step in range(150):
        d = Device(m)
        what = g.choice(["advance", "advance", "fork", "compact"])
        if what == "advance":
            counts = [int(x) for x in g.integers(0, 3 * page, batch)]
            window = int(g.choice([0, 40]))
            got, want = d.advance(counts, window, 4, bool(step % 2)), m.advance(counts, window, 4)
            same(got, want, f"step {step}")
            m.table, m.uses = want[0], want[1]
            m.lens = np.minimum(m.lens + np.array(counts, np.int32), per * page)
        elif what == "fork":
            parents = [int(x) for x in g.integers(-1, batch, batch)]
            got, want = d.fork(parents, bool(step % 2)), m.fork(parents)
            same(got, want, f"step {step}")
            m.table, m.lens, m.uses = want[0], want[1], want[2]
        else:
            got, want = d.compact(bool(step % 2)), m.compact()
            same(got, want, f"step {step}")
            m.table, m.uses = want[0], want[1]
            assert (m.uses[:want[3]] > 0).all() and not m.uses[want[3]:].any()
        named = np.bincount(m.table[m.table >= 0], minlength=P)
        assert np.array_equal(named, m.uses)
        for b in range(batch):  # what is still written has one user
            written = m.table[b, m.lens[b] // page:]
            assert (m.uses[written[written >= 0]] == 1).all()
