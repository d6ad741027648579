"""The chunk kernel's ring of code tiles, replayed on the host: the kernel's own index arithmetic
(csrc/attn_index.h, compiled here) with every copy, conversion warp and product at a pace of its own.
Each reader has to find its own tile, whole, wherever the others are."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "moe_expert_layer_sigmoid_gb300", "csrc")
RAWS, SLOTS, SCALES, WARPS = 3, 3, 4, 4   # tiles of codes, bf16 tiles, scale slots, warps of a group

SOURCE = """
#include "attn_index.h"
using R = moe::CodeRing<%d>;
extern "C" {
uint32_t slot(uint32_t it) { return R::slot(it); }
uint32_t full(uint32_t it) { return R::full(it); }
uint32_t full_parity(uint32_t it) { return R::full_parity(it); }
uint32_t free_parity(uint32_t it) { return R::free_parity(it); }
uint32_t fulls() { return R::kFull; }
}
""" % RAWS


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    src, lib = str(d / "ring.cpp"), str(d / "ring.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib], check=True)
    L = ctypes.CDLL(lib)
    for n in ("slot", "full", "full_parity", "free_parity", "fulls"):
        getattr(L, n).restype = ctypes.c_uint32
    return L


class OneBarrierToASlot:
    """The indexing that cannot work: both groups wait on one barrier of a slot."""
    slot = staticmethod(lambda it: it % RAWS)
    full = staticmethod(lambda it: it % RAWS)
    full_parity = staticmethod(lambda it: it // RAWS & 1)
    free_parity = staticmethod(lambda it: it // RAWS & 1 ^ 1)
    fulls = staticmethod(lambda: RAWS)


class Barrier:
    """An mbarrier: a phase ends when its arrivals and its bytes (here: copies) are all in."""

    changes = 0

    def __init__(self, count):
        self.count = self.pending = count
        self.phase = self.tx = 0

    def _turn(self):
        Barrier.changes += 1
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self):
        assert self.pending > 0, "an arrival too many"
        self.pending -= 1
        self._turn()

    def expect(self):
        self.tx += 1
        self.arrive()

    def landed(self):
        self.tx -= 1
        self._turn()

    def done(self, parity):
        """try_wait.parity: the phase before the current one has this parity."""
        return (self.phase - 1) & 1 == parity


def replay(ring, tiles, split, seed, slow):
    """One stretch of `tiles` key tiles; `slow` scales the copies of keys (0), values (1) or random ones."""
    rng = random.Random(seed)
    now, events = 0, []        # (time, order, function)

    def later(dt, fn):
        events.append((now + dt, len(events) + rng.random(), fn))

    rawf = [Barrier(1) for _ in range(ring.fulls())]
    rawe = [Barrier(WARPS) for _ in range(RAWS)]
    full = [Barrier(WARPS) for _ in range(SLOTS)]
    empty = [Barrier(1) for _ in range(SLOTS)]
    raw, flying = [None] * RAWS, [None] * RAWS     # codes in place, copy in flight
    bf, using = [[None] * WARPS for _ in range(SLOTS)], [None] * SLOTS
    scale = [[None, None] for _ in range(SCALES)]

    def copies():
        for it in range(2 * tiles):
            s, kv, j = ring.slot(it), it & 1, it // 2
            while not rawe[s].done(ring.free_parity(it)):
                yield 0
            assert flying[s] is None, "a copy into a slot that another is on its way to"
            flying[s] = it
            b = rawf[ring.full(it)]
            b.expect()

            def land(s=s, it=it, kv=kv, j=j, b=b):
                raw[s], flying[s] = it, None
                scale[j % SCALES][kv] = j
                b.landed()
            late = slow == kv or slow == 2 and rng.random() < 0.2
            later(rng.uniform(1, 60) if late else rng.uniform(1, 3), land)
            yield rng.uniform(0, 0.3)

    def conversion(kv, warp):
        for it in range(kv, 2 * tiles, 2):
            s, sl, j = ring.slot(it), it % SLOTS, it // 2
            while not rawf[ring.full(it)].done(ring.full_parity(it)):
                yield 0
            while not empty[sl].done(it // SLOTS & 1 ^ 1):
                yield 0
            assert raw[s] == it and flying[s] is None, f"the codes of copy {raw[s]} taken for those of {it}"
            assert scale[j % SCALES][kv] == j, "a scale that is not there"
            yield rng.uniform(0.5, 1.5)
            assert raw[s] == it and flying[s] is None, "codes overwritten while they are read"
            assert using[sl] is None, "a tile overwritten before its product is done"
            bf[sl][warp] = it
            full[sl].arrive()
            rawe[s].arrive()

    def tile_ready(it):
        while not full[it % SLOTS].done(it // SLOTS & 1):
            yield 0
        assert bf[it % SLOTS] == [it] * WARPS, "a product of another tile"
        using[it % SLOTS] = it

    def released(it):
        def done():
            using[it % SLOTS] = None
            empty[it % SLOTS].arrive()
        later(rng.uniform(0.1, 2.0), done)

    def products():
        """Scores of tile i, softmax (which reads the scales), values of tile i, as the kernel orders them."""
        ahead = 2 if split else 1
        for i in range(min(ahead, tiles)):
            yield from tile_ready(2 * i)
            released(2 * i)
        for i in range(tiles):
            yield from tile_ready(2 * i + 1)
            yield rng.uniform(0.2, 2.0)
            assert scale[i % SCALES] == [i, i], "scales overwritten while they are read"
            released(2 * i + 1)
            if i + ahead < tiles:
                yield from tile_ready(2 * (i + ahead))
                released(2 * (i + ahead))

    agents = [copies(), products()] + [conversion(kv, w) for kv in (0, 1) for w in range(WARPS)]
    wake = {a: 0.0 for a in agents}
    for _ in range(4000 * tiles):
        if not wake:
            return
        ready = sorted((e for e in events if e[0] <= now), key=lambda e: e[:2])
        for e in ready:
            events.remove(e)
            e[2]()
        moved, before = False, Barrier.changes
        for a in rng.sample(list(wake), len(wake)):
            if wake[a] <= now:
                try:
                    dt = next(a)
                    wake[a] = now + dt
                    moved |= dt > 0
                except StopIteration:
                    del wake[a]
                    moved = True
        if not ready and not moved and Barrier.changes == before:
            nxt = [e[0] for e in events] + [t for t in wake.values() if t > now]
            assert nxt, "everyone waits"
            now = min(nxt)
    raise AssertionError("no end")


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("slow", [0, 1, 2, None])
def test_each_reader_finds_its_own_tile(ring, slow, split):
    for seed in range(12):
        replay(ring, 1 + seed * 2, split, seed, slow)


@pytest.mark.parametrize("slow", [0, 1, 2])
def test_the_replay_sees_a_shared_barrier(slow):
    with pytest.raises(AssertionError, match="taken for|not there|in flight|overwritten|too many|on its way|everyone"):
        for seed in range(40):
            replay(OneBarrierToASlot, 20, False, seed, slow)


def test_each_barrier_has_one_group_and_all_its_phases(ring):
    seen = {}
    for it in range(600):
        seen.setdefault(ring.full(it), []).append((it & 1, ring.full_parity(it)))
    assert sorted(seen) == list(range(ring.fulls()))
    for visits in seen.values():
        assert len({kv for kv, _ in visits}) == 1
        assert [p for _, p in visits] == [i & 1 for i in range(len(visits))]
