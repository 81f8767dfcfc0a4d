"""Upkeep of pools of more than a million pages (bookkeeping alone, no keys and values), whose counts of
free pages take several turns of a workgroup to sum and to search: against plain Python."""
import numpy as np
import pytest

from test_gpu_attn import _case
from test_gpu_pages import Device, Model, same

pytestmark = pytest.mark.gpu

TURN = 256 * 4096  # pages whose counts a workgroup takes in one turn


def free_pages(kind, P, g):
    if kind == "across a turn":
        return np.arange(TURN - 400, min(P, TURN + 1800))
    if kind == "past it":
        return np.sort(g.choice(np.arange(TURN, P), 2500, replace=False))
    if kind == "ends":  # a few in front of it, the last page of the pool
        return np.unique(np.concatenate([[0, 4095, 4096, TURN - 1, TURN, P - 1], g.choice(P, 1200)]))
    return np.array([P - 1])


def cache(kind, P, batch, per, page=16):
    g = np.random.default_rng(P % 1000 + len(kind))
    uses = g.integers(1, 4, P).astype(np.int32)  # most are held by streams that are not here
    free = free_pages(kind, P, g)
    uses[free] = g.choice([0, 0, -2], len(free))
    table = np.full((batch, per), -1, np.int32)
    lens = g.integers(0, 40 * page, batch).astype(np.int32) | 1  # a partly filled page each, for a fork to copy
    for b in range(batch):
        held = -(-int(lens[b]) // page)
        table[b, :held] = g.choice(np.flatnonzero(uses > 0), held)
        table[b, held:held + 5] = g.choice([-1, P, -9], 5)
    np.add.at(uses, table[(table >= 0) & (table < P)], 1)
    return Model(table, lens, uses, page)


POOLS = [TURN + 1, TURN + 4097, 2 * TURN + 5000]
KINDS = ["across a turn", "past it", "ends", "the last page"]


@pytest.mark.parametrize("P", POOLS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("in_place", [False, True])
def test_advance(P, kind, in_place):
    _case(f"advance {P} pages, free ones {kind}, in place {in_place}")
    if kind == "past it" and P < TURN + 2500:
        P += 2500
    m = cache(kind, P, 4, 3000)
    for counts in ([1, 300 * 16, 1500 * 16 + 3, 40 * 16], [2400 * 16, 16, 0, 5]):
        same(Device(m).advance(counts, 0, 0, in_place), m.advance(counts), f"{counts}")


@pytest.mark.parametrize("P", POOLS[1:])
@pytest.mark.parametrize("kind", KINDS)
def test_fork(P, kind):
    _case(f"fork {P} pages, free ones {kind}")
    m = cache(kind, P, 700, 64)
    for parents in ([3] * 700, [b // 3 for b in range(700)]):
        same(Device(m).fork(parents), m.fork(parents), "fork")


@pytest.mark.parametrize("P", POOLS[1:])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(P, kind, in_place):
    _case(f"compact {P} pages, free ones {kind}, in place {in_place}")
    m = cache(kind, P, 3, 100)
    same(Device(m).compact(in_place), m.compact(), "compact")
