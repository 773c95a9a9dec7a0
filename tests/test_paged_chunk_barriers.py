"""A model of the barriers of paged_chunk_kernel (paged_chunk.cuh), run under
random schedules on the host.

A wait on an mbarrier sees only the parity of its phase.  The model's barriers
count their phases, and a wait that passes although another phase than its own
is the last one complete fails the test; so does a schedule that comes to a
stop, an arrival too many, and a copy or MMA still under way when every warp of
the pair is done.  Sizes and warps are those of the source.  A form with one
ring of slots for S and PV together, which parity cannot tell apart, is found
out by the same model."""
import os
import random
import re
from collections import deque

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_latent_space_lca_b200", "csrc",
                      "paged_chunk.cuh")


def constants():
    """The integer constants that paged_chunk.cuh gives as numbers."""
    out = {}
    with open(SOURCE) as f:
        for line in f:
            if line.startswith("constexpr int"):
                out.update((k, int(v)) for k, v in re.findall(r"(PC_\w+) = (\d+)\s*[,;]", line))
    return out


C = constants()
KS, VS = C["PC_KS"], C["PC_VS"]                       # slots of a cache tile for S, for PV
KRING, VRING = C["PC_KRING"], C["PC_VRING"]
KWARPS, VWARPS, SOFTMAX = C["PC_KWARPS"], C["PC_VWARPS"], C["PC_SOFTMAX"]


class Aliased(AssertionError):
    pass


class Bar:
    def __init__(self, count):
        self.count = self.pending = count
        self.bytes = self.phase = 0

    def arrive(self, expect=0):
        assert self.pending > 0, "an arrival too many"
        self.pending -= 1
        self.bytes += expect
        self._turn()

    def complete(self):   # one copy's bytes
        self.bytes -= 1
        self._turn()

    def _turn(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase += 1
            self.pending = self.count

    def done(self, k):
        """Phase k (-1: the one before the first) as a parity wait sees it."""
        if (self.phase & 1) == (k & 1):
            return False
        if self.phase != k + 1:
            raise Aliased(f"phase {k} waited for, {self.phase} complete")
        return True


class Pair:
    """Two CTAs on the same pieces: (cache tiles, PV slots of the last one,
    edge tiles at the end) each."""

    def __init__(self, pieces, seed, one_ring=0):
        self.pieces, self.rng = pieces, random.Random(seed)
        # the places that each cache tile's slots take in their ring's order
        self.k_places, self.v_places = [], []
        nk = nv = 0
        for tiles, last, _ in pieces:
            for i in range(tiles):
                n = last if i + 1 == tiles else VS
                k0, v0 = (nk + nv, nk + nv + KS) if one_ring else (nk, nv)
                self.k_places.append(list(range(k0, k0 + KS)))
                self.v_places.append(list(range(v0, v0 + n)))
                nk, nv = nk + KS, nv + n
        self.k_ring, self.v_ring = (one_ring, one_ring) if one_ring else (KRING, VRING)
        self.kfull = [Bar(1) for _ in range(self.k_ring)]
        self.kempty = [[Bar(1) for _ in range(self.k_ring)] for _ in range(2)]
        self.vfull = self.kfull if one_ring else [Bar(1) for _ in range(self.v_ring)]
        self.vempty = self.kempty if one_ring else [[Bar(1) for _ in range(self.v_ring)] for _ in range(2)]
        two = lambda count: [Bar(count), Bar(count)]  # noqa: E731
        self.qfull, self.oread = Bar(1), Bar(2 * SOFTMAX)
        self.sdone, self.vdone = [two(1), two(1)], [two(1), two(1)]   # [CTA][n & 1]
        self.sread, self.pfull = two(2 * SOFTMAX), two(2 * SOFTMAX)
        self.vready = two(1)                                           # [CTA]
        self.pairs = [[Bar(2) for _ in range(SOFTMAX // 2)] for _ in range(2)]
        self.loose = []                      # copies and remote arrivals: land in any order
        self.chains = {"S": deque(), "PV": deque()}   # commits of one issuing thread: in order
        fetch = []
        for cta in range(2):
            if one_ring:   # each of four producers brings every fourth slot, for S or for PV
                both = [k + v for k, v in zip(self.k_places, self.v_places)]
                fetch += [self.producer(cta, both, self.kfull, self.kempty[cta], p, 4, p == 0) for p in range(4)]
            else:
                fetch += [self.producer(cta, self.k_places, self.kfull, self.kempty[cta], p, KWARPS, p == 0)
                          for p in range(KWARPS)]
                fetch += [self.producer(cta, self.v_places, self.vfull, self.vempty[cta], p, VWARPS, False)
                          for p in range(VWARPS)]
        self.warps = fetch + [self.s_warp(), self.pv_warp()]
        self.warps += [self.softmax(c, w) for c in range(2) for w in range(SOFTMAX)]

    # ---- the roles: each yields a condition to wait for, or None for a pause
    def producer(self, cta, places, full, empty, p, step, queries):
        ring, n, mine = len(full), 0, []
        for tiles, _, _ in self.pieces:
            if queries:
                if n > 0:
                    yield lambda k=n - 1: self.sdone[cta][k & 1].done(k >> 1)
                if cta == 0:
                    self.qfull.arrive(2)
                self.loose.append(self.qfull.complete)
            for n in range(n, n + tiles):
                for x in (x for x in places[n] if x % step == p):
                    mine.append(x)
                    yield lambda x=x: empty[x % ring].done(x // ring - 1)
                    if cta == 0:
                        full[x % ring].arrive(2)
                    self.loose.append(full[x % ring].complete)
                    yield None
            n += 1
        for x in reversed(mine):   # the ring's last uses
            if x + ring <= places[-1][-1]:
                break
            if cta == 0:
                yield lambda x=x: full[x % ring].done(x // ring)
            yield lambda x=x: empty[x % ring].done(x // ring)

    def commit(self, chain, bars):   # to both CTAs
        self.chains[chain].extend(b.arrive for b in bars)

    def s_warp(self):
        n = 0
        for piece, (tiles, _, _) in enumerate(self.pieces):
            yield lambda k=piece: self.qfull.done(k)
            for n in range(n, n + tiles):
                yield lambda k=n: self.sread[k & 1].done((k >> 1) - 1)
                for x in self.k_places[n]:
                    yield lambda x=x: self.kfull[x % self.k_ring].done(x // self.k_ring)
                    self.commit("S", [e[x % self.k_ring] for e in self.kempty])
                self.commit("S", [d[n & 1] for d in self.sdone])
            n += 1
        yield lambda k=n - 1: self.sread[k & 1].done(k >> 1)

    def pv_warp(self):
        n = 0
        for piece, (tiles, _, edges) in enumerate(self.pieces):
            for i in range(tiles):
                if i >= tiles - edges:
                    for x in self.v_places[n]:
                        yield lambda x=x: self.vfull[x % self.v_ring].done(x // self.v_ring)
                    self.vready[0].arrive()
                    self.loose.append(self.vready[1].arrive)
                if i == 0:
                    yield lambda k=piece - 1: self.oread.done(k)
                yield lambda k=n: self.pfull[k & 1].done(k >> 1)
                for x in self.v_places[n]:
                    yield lambda x=x: self.vfull[x % self.v_ring].done(x // self.v_ring)
                    self.commit("PV", [e[x % self.v_ring] for e in self.vempty])
                self.commit("PV", [d[n & 1] for d in self.vdone])
                n += 1
        yield lambda k=len(self.pieces) - 1: self.oread.done(k)

    def softmax(self, cta, warp):
        swap = self.pairs[cta][warp % (SOFTMAX // 2)]
        n = edge = swaps = 0

        def exchange():   # a named barrier, which counts
            nonlocal swaps
            swaps += 1
            swap.arrive()
            return lambda k=swaps: swap.phase >= k

        for tiles, _, edges in self.pieces:
            for i in range(tiles):
                yield lambda k=n: self.sdone[cta][k & 1].done(k >> 1)
                self.loose.append(self.sread[n & 1].arrive)
                is_edge, early = i >= tiles - edges, self.rng.random() < 0.5   # early: rows to clear
                if is_edge and early:
                    yield lambda k=edge: self.vready[cta].done(k)
                yield exchange()
                if n > 0:
                    yield lambda k=n - 1: self.vdone[cta][k & 1].done(k >> 1)
                if is_edge and not early:
                    yield lambda k=edge: self.vready[cta].done(k)
                edge += is_edge
                yield None
                self.loose.append(self.pfull[n & 1].arrive)
                n += 1
            yield exchange()
            yield lambda k=n - 1: self.vdone[cta][k & 1].done(k >> 1)
            yield None
            self.loose.append(self.oread.arrive)

    # ---- one random schedule: some warps, copies or MMAs much slower than others
    def run(self):
        rng = self.rng
        waiting = {w: None for w in self.warps}
        speed = {w: rng.choice([0.02, 0.2, 1, 5]) for w in self.warps}
        loose_speed, mma_speed = rng.choice([0.05, 0.5, 3]), rng.choice([0.05, 0.5, 3])
        while waiting:
            agents = list(waiting) + ["loose", "S", "PV"]
            weights = [speed[w] for w in waiting] + [loose_speed * min(len(self.loose), 6), mma_speed, mma_speed]
            assert self._can_move(waiting), f"{len(waiting)} warps wait for one another"
            for agent in rng.choices(agents, weights, k=24):
                self._move(agent, waiting)
        assert not self.loose and not self.chains["S"] and not self.chains["PV"], "work under way at the end"

    def _can_move(self, waiting):
        return (self.loose or self.chains["S"] or self.chains["PV"]
                or any(cond is None or cond() for cond in waiting.values()))

    def _move(self, agent, waiting):
        if agent == "loose":
            if self.loose:
                self.loose.pop(self.rng.randrange(len(self.loose)))()
        elif agent in ("S", "PV"):
            if self.chains[agent]:
                self.chains[agent].popleft()()
        elif agent in waiting and (waiting[agent] is None or waiting[agent]()):
            try:
                waiting[agent] = next(agent)
            except StopIteration:
                del waiting[agent]


def some_pieces(rng):
    """One to five query tiles of a cluster's range, short and long."""
    out = []
    for _ in range(rng.randint(1, 5)):
        tiles = rng.choice([1, 1, 1, 2, 3, 6])
        out.append((tiles, rng.randint(1, VS), rng.randint(0, min(tiles, 2))))
    return out


@pytest.mark.parametrize("first", range(0, 120, 20))
def test_barriers_under_random_schedules(first):
    for seed in range(first, first + 20):
        Pair(some_pieces(random.Random(seed)), seed).run()


def test_one_ring_for_both_consumers_is_found_out():
    found = 0
    for seed in range(40):
        try:
            Pair([(6, VS, 1), (4, VS, 1)], seed, one_ring=15).run()
        except Aliased:
            found += 1
    assert found > 0


def test_constants_are_read():
    assert min(KS, VS, KRING, VRING, KWARPS, VWARPS, SOFTMAX) > 0
    assert KS % KWARPS == 0 and VS % VWARPS == 0 and VS <= VRING
