"""Host model of the rotary kernel's ring (rotary_kernel): a producer warp and the turning warps of a CTA as generators that
wait on and arrive at mbarriers with the kernel's counts and wait parities.  Copies in land, and copies out read their stage,
in any order at random moments.  Every run must finish, never poll a barrier two phases away from the phase it waits for,
never write a stage that is still read, and turn and copy out each token once.

A copy that never lands makes the waits that depend on it give up, as the kernel's bounded waits do: the roles must end all
the same, and no other copy may still be landing when they have.

Tests plant mistakes that the model must report.  No GPU is involved.
"""
import random
import re

import pytest

from _kernel_consts import _source, kconst

FILE = "rotary.cu"
TEXT = _source(FILE)
STAGES, WARPS = kconst("kRoStages", FILE), kconst("kRoWarps", FILE)


def count(barrier):
    e = re.search(r"mbar_init\(&" + barrier + r"\[\w\], ([^)]+)\)", TEXT).group(1)
    return int(e) if e.isdigit() else kconst(e, FILE)


def last_fills(out, n):
    """Fills of each stage that the producer waits for after a wait that gave up, by the kernel's expressions: `out` of n
    tokens have been copied out."""
    e = re.search(r"const int filled = ([^;]+);", TEXT).group(1)
    filled = eval(e, {"out": out, "n": n, "kRoStages": STAGES, "min": min})
    e = re.search(r"const int fills = ([^;]+);", TEXT).group(1).replace("/", "//")
    assert "filled" in e
    return [eval(e, {"filled": filled, "s": s, "kRoStages": STAGES}) for s in range(STAGES)]


def marks():
    """Whether the producer's branch behind a wait that gave up marks the rows of the tokens that were not copied out."""
    a = TEXT.index("    if (!ok)")
    return "for (int j = out; j < n; ++j) ro_mark(a.q_out, geo.q_bytes, a.k_out, geo.k_bytes, token(j));" in \
        TEXT[a:TEXT.index("bulk_wait_all();", a)]


class Bar:
    def __init__(self, n):
        self.n, self.pending, self.done = n, n, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.done, self.pending = self.done + 1, self.n


class Sim:
    def __init__(self, tokens, rng, mistake=None, lost=None):
        self.n, self.rng, self.mistake, self.lost = tokens, rng, mistake, lost
        self.full, self.done = ([Bar(count(b)) for _ in range(STAGES)] for b in ("full", "done"))
        self.stage = [None] * STAGES         # (token, warps that have turned it)
        self.table = [None] * STAGES         # the token whose angles a stage holds
        self.readers = [0] * STAGES
        self.loads, self.copies = [], []     # (stage, token) on its way in; a copy out
        self.out, self.nan = [], []          # tokens copied out, tokens whose rows are marked

    def wait(self, bar, need, token):
        """Until `need` phases are done, seen as the kernel sees them: by the parity of the last of them.  `token`: whose
        copy or turning that is."""
        parity = (need - 1) & 1

        def ok():
            assert need - 1 <= bar.done <= need, f"{bar.done} phases done, waiting for {need}"
            return (bar.done & 1) != parity
        ok.doomed = self.lost is not None and token >= self.lost
        return ok

    def producer(self):
        filled, out, ok = 0, 0, True
        for i in range(self.n + STAGES):
            s = i % STAGES
            if i >= STAGES and i - STAGES < self.n:
                if self.mistake != "early copy":
                    ok = yield self.wait(self.done[s], (i - STAGES) // STAGES + 1, i - STAGES)
                if not ok:
                    break
                self.copies.append((s, i - STAGES))
                out += 1
            if i >= self.n:
                continue
            assert not self.readers[s] or self.mistake, "a table rewritten while it is read"
            self.table[s] = i
            if self.mistake != "refill":
                while self.copies:  # (their reads: not a bounded wait)
                    yield lambda: not self.copies
            assert not self.readers[s] and all(x != s for x, _ in self.copies), "a stage filled while it is read"
            self.loads.append((s, i))
            filled += 1
        if not ok:
            for s, fills in enumerate(last_fills(out, self.n)):
                if fills > 0 and self.mistake != "no last wait":
                    assert fills == len(range(s, filled, STAGES)), f"stage {s}: waits for fill {fills}"
                    last = self.wait(self.full[s], fills, 0)
                    last.doomed = s + (fills - 1) * STAGES == self.lost
                    yield last
            self.nan += range(out, self.n) if marks() else []
        while self.copies:  # (not a bounded wait either)
            yield lambda: not self.copies

    def turner(self, w):
        for i in range(self.n):
            s = i % STAGES
            if not (yield self.wait(self.full[s], (i + (1 if self.mistake == "phase" else 0)) // STAGES + 1, i)):
                return
            assert self.stage[s][0] == i and self.table[s] == i, f"token {i}: stage {self.stage[s]}, angles of {self.table[s]}"
            self.readers[s] += 1
            yield None
            self.stage[s][1] += 1
            self.readers[s] -= 1
            self.done[s].arrive()

    def run(self):
        roles = [self.producer()] + [self.turner(w) for w in range(WARPS)]
        soon = self.rng.choice([0.1, 0.95])
        blocked, live, begun, steps = [None] * len(roles), set(range(len(roles))), set(), 0
        while live or self.copies or any(t != self.lost for _, t in self.loads):
            steps += 1
            assert steps < 100000, "no progress"
            if not live:
                assert not self.loads or all(t == self.lost for _, t in self.loads), "a copy lands after the CTA's end"
            moves = [("role", r) for r in live if blocked[r] is None or blocked[r]()]
            moves += [("land", x) for x in self.loads if x[1] != self.lost] + [("copy", x) for x in self.copies]
            # a bounded wait for the lost copy, or for what follows from it, runs out at any moment
            doomed = [("role", r) for r in live if blocked[r] and getattr(blocked[r], "doomed", False)]
            gave_up = doomed and (not moves or self.rng.random() < soon)
            moves = doomed if gave_up else moves
            assert moves, "deadlock"
            kind, x = self.rng.choice(moves)
            if kind == "land":
                self.loads.remove(x)
                s, t = x
                assert not self.readers[s], "a copy lands in a stage that is read"
                self.stage[s] = [t, 0]
                self.full[s].arrive()
            elif kind == "copy":
                self.copies.remove(x)
                s, t = x
                assert self.stage[s] == [t, WARPS], f"token {t} copied out of {self.stage[s]}"
                self.out.append(t)
            else:
                try:
                    blocked[x] = roles[x].send(not gave_up if x in begun else None)
                    begun.add(x)
                except StopIteration:
                    live.discard(x)
        return self


@pytest.mark.parametrize("seed", range(20))
def test_random_schedules(seed):
    rng = random.Random(seed)
    n = rng.randint(1, 30)
    assert sorted(Sim(n, rng).run().out) == list(range(n))


@pytest.mark.parametrize("mistake", ["early copy", "refill", "phase"])
def test_planted_mistakes_are_reported(mistake):
    reported = 0
    for seed in range(20):
        try:
            Sim(20, random.Random(seed), mistake).run()
        except AssertionError:
            reported += 1
    assert reported >= 10, f"{mistake}: reported in {reported} of 20 runs"


@pytest.mark.parametrize("seed", range(20))
def test_a_copy_that_never_lands_ends_every_role(seed):
    # the last fill of every stage is waited for, whichever wait gave up first
    rng = random.Random(seed)
    n = rng.randint(1, 30)
    lost = rng.randrange(n)
    out = Sim(n, rng, lost=lost).run().out
    assert sorted(out) == list(range(len(out))) and len(out) <= lost


def test_an_end_without_the_last_wait_is_reported():
    reported = 0
    for seed in range(40):
        rng = random.Random(seed)
        try:
            Sim(20, rng, "no last wait", lost=rng.randrange(16)).run()
        except AssertionError:
            reported += 1
    assert reported >= 10, f"reported in {reported} of 40 runs"


@pytest.mark.parametrize("seed", range(20))
def test_a_token_that_was_not_copied_out_is_marked(seed):
    # no row is left as it was: it is turned, or NaN
    rng = random.Random(seed)
    n = rng.randint(1, 30)
    sim = Sim(n, rng, lost=rng.randrange(n)).run()
    assert sorted(sim.out + sim.nan) == list(range(n))
    assert not Sim(n, rng).run().nan
