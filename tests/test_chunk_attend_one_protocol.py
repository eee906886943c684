"""Host model of the chunk attention's one-token items (ca_one_produce and ca_one_attend): the producer warp and the eight
computing warps of a CTA as generators that wait on and arrive at mbarriers with the kernel's counts and wait parities.  Copies
land in any order at random moments.  Over an E4M3 cache a block's K and V share a place, and every warp passes every place;
over a bf16 cache they have one each.  At an item's end the warps' sums meet in shared memory.

Random lists of items (1 to 9 blocks) run under random schedules.  Every run must finish, never poll a barrier two phases away
from the phase it waits for, never write a place, a page flag or a sum that is still to be read, and read in every use what it
expects.  Tests plant mistakes that the model must report.  No GPU is involved.
"""
import random
import re

import pytest

from _kernel_consts import _source, kconst

FILE = "chunk_attend.cu"
TEXT = _source(FILE)
INFO, PLACES, WARPS = kconst("kCaInfo", FILE), kconst("kCaOnePlaces", FILE), 8


def count(barrier):
    return int(re.search(r"mbar_init\(&sm\." + barrier + r"(?:\[\w\])?, (\d+)\)", TEXT).group(1))


class Bar:
    def __init__(self, n):
        self.n, self.pending, self.done = n, n, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.done, self.pending = self.done + 1, self.n


class Sim:
    def __init__(self, items, fp8, rng, mistake=None):
        self.items, self.fp8, self.rng, self.mistake = items, fp8, rng, mistake
        self.bar = {(b, i): Bar(count(b)) for b, n in (("one_full", PLACES), ("one_empty", PLACES), ("one_info_full", INFO),
                                                       ("one_info_empty", INFO), ("one_x_full", 1), ("one_x_done", 1))
                    for i in range(n)}
        self.info, self.place, self.flag = [None] * INFO, [None] * PLACES, [None] * PLACES
        self.unread = [0] * PLACES           # warps that have not given the place back
        self.loads = []
        self.sums, self.readers = [None] * WARPS, [0] * WARPS
        self.joined = []

    def wait(self, b, i, need):
        """Until `need` phases are done, seen as the kernel sees them: by the parity of the last of them."""
        bar, parity = self.bar[b, i], (need - 1) & 1

        def ok():
            assert need - 1 <= bar.done <= need, f"{b}{i}: {bar.done} phases done, waiting for {need}"
            return (bar.done & 1) != parity
        return ok

    def arrive(self, b, i=0):
        self.bar[b, i].arrive()

    def producer(self):
        place = 0
        for n, nb in enumerate(self.items + [0]):
            yield self.wait("one_info_empty", n % INFO, n // INFO)
            self.info[n % INFO] = (n, nb)
            self.arrive("one_info_full", n % INFO)
            for b in range(nb):
                for kind in ("KV",) if self.fp8 else ("K", "V"):
                    s = place % PLACES
                    yield self.wait("one_empty", s, place // PLACES)
                    assert not self.unread[s], f"place {s} written while {self.place[s]} is read"
                    self.flag[s] = (n, b)
                    self.unread[s] = WARPS
                    self.loads.append((s, (n, b, kind)))
                    place += 1

    def use(self, s, tag):
        assert self.place[s] == tag, f"place {s} holds {self.place[s]}, expected {tag}"

    def release(self, s):
        self.unread[s] -= 1
        self.arrive("one_empty", s)

    def attend(self, w):
        place = 0
        turns = PLACES - 1 if self.mistake == "phase" else PLACES
        for n in range(len(self.items) + 1):
            yield self.wait("one_info_full", n % INFO, n // INFO + 1)
            item, nb = self.info[n % INFO]
            assert item == n
            self.arrive("one_info_empty", n % INFO)
            if nb == 0:
                return
            for b in range(nb):
                s = place % PLACES
                yield self.wait("one_full", s, place // turns + 1)
                assert self.flag[s] == (n, b), f"flag of {self.flag[s]}, expected {(n, b)}"
                place += 1
                if self.fp8:
                    if place & 1 == w >> 2:
                        if self.mistake == "early":
                            self.release(s)
                        yield None
                        self.use(s, (n, b, "KV"))
                    if self.mistake != "early" or place & 1 != w >> 2:
                        self.release(s)
                    continue
                self.use(s, (n, b, "K"))
                yield None
                self.use(s, (n, b, "K"))
                self.release(s)
                v = place % PLACES
                if self.mistake != "no wait":
                    yield self.wait("one_full", v, place // turns + 1)
                place += 1
                self.use(v, (n, b, "V"))
                yield None
                self.use(v, (n, b, "V"))
                self.release(v)
            # the warps' sums meet; each warp joins two rows of all of them
            assert not self.readers[w], f"the sums of warp {w} rewritten while they are read"
            self.sums[w] = n
            yield None
            self.arrive("one_x_full")
            yield self.wait("one_x_full", 0, n + 1)
            for x in range(WARPS):
                assert self.sums[x] == n, f"sums of item {self.sums[x]}, expected {n}"
                self.readers[x] += 1
            yield None
            for x in range(WARPS):
                self.readers[x] -= 1
            self.joined.append((n, w))
            self.arrive("one_x_done")
            if self.mistake != "no end":
                yield self.wait("one_x_done", 0, n + 1)

    def run(self):
        roles = [self.producer()] + [self.attend(w) for w in range(WARPS)]
        blocked, live, steps = [None] * len(roles), set(range(len(roles))), 0
        while live or self.loads:
            steps += 1
            assert steps < 200000, "no progress"
            moves = [("role", r) for r in live if blocked[r] is None or blocked[r]()] + [("land", x) for x in self.loads]
            assert moves, "deadlock"
            kind, x = self.rng.choice(moves)
            if kind == "land":
                self.loads.remove(x)
                self.place[x[0]] = x[1]
                self.arrive("one_full", x[0])
            else:
                try:
                    blocked[x] = next(roles[x])
                except StopIteration:
                    live.discard(x)
        assert sorted(self.joined) == [(n, w) for n in range(len(self.items)) for w in range(WARPS)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seed", range(12))
def test_random_schedules(seed, fp8):
    rng = random.Random(seed)
    Sim([rng.randint(1, 9) for _ in range(rng.randint(0, 12))], fp8, rng).run()


@pytest.mark.parametrize("mistake,fp8", [("phase", False), ("phase", True), ("early", True), ("no wait", False),
                                         ("no end", False), ("no end", True)])
def test_planted_mistakes_are_reported(mistake, fp8):
    reported = 0
    for seed in range(20):
        rng = random.Random(seed)
        try:
            Sim([rng.randint(1, 3) for _ in range(24)], fp8, rng, mistake).run()
        except AssertionError:
            reported += 1
    assert reported >= 10, f"{mistake}: reported in {reported} of 20 runs"
