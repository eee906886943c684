"""Host model of the chunk attention's synchronisation (chunk_attend_kernel, the items of two tiles and of one).

The producer warp, the MMA thread, eight softmax warps and (over an E4M3 cache) four widening warps are generators that
wait on and arrive at mbarriers with the kernel's counts and wait parities.  Copies land in any order at random moments;
the tensor cores execute the issued products and commits in order, some time after they were issued.  Random lists of
pieces (1 to 16 tokens, 1 to 7 blocks) run under random schedules.  Every run must finish, never poll a barrier two phases
away from the phase it waits for, never write a place that is still read, and read in every use the tile, the scores, the
weights and the sums that it expects.

Tests plant mistakes that the model must report: a K place given back by the first of its two readers, a wait that takes
the phase of a ring of two places as if it had four, scores issued before the weights that lie over them are used, and
sums read without the wait for their last product.  No GPU is involved.
"""
import random
import re

import pytest

from _kernel_consts import _source, kconst

FILE = "chunk_attend.cu"
TEXT = _source(FILE)
INFO = kconst("kCaInfo", FILE)


def shape(name, fp8):
    """`static constexpr int <name> = kFp8 ? a : b;`"""
    m = re.search(r"static constexpr int " + name + r" = kFp8 \? (\d+) : (\d+);", TEXT)
    return int(m.group(1 if fp8 else 2))


def count(barrier, fp8):
    """Arrival count of `mbar_init(&sm.<barrier>[..], <count>)`: a number, a choice by the cache, or one with the widening warps."""
    e = re.search(r"mbar_init\(&sm\." + barrier + r"(?:\[\w\])?, ([^)]+)\)", TEXT).group(1)
    m = re.fullmatch(r"kFp8 \? (\d+) : (\d+)", e)
    if m:
        return int(m.group(1 if fp8 else 2))
    return eval(e.replace("Shape::kWiden", str(shape("kWiden", fp8))))


class Bar:
    def __init__(self, name, n):
        self.name, self.n, self.pending, self.done = name, n, n, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0, self.name
        if self.pending == 0:
            self.done, self.pending = self.done + 1, self.n


class Sim:
    def __init__(self, items, fp8, rng, mistake=None):
        self.items, self.fp8, self.rng, self.mistake = items, fp8, rng, mistake
        self.T, self.R, self.W = (shape(n, fp8) for n in ("kTiles", "kRaw", "kWiden"))
        sizes = {"q_full": 2, "q_ready": 2, "q_empty": 2, "kv_full": self.T, "kv_empty": self.T, "raw_full": self.R,
                 "raw_empty": self.R, "s_full": 2, "p_full": 2, "o_full": 2, "info_full": INFO, "info_empty": INFO,
                 "x_full": 1, "x_done": 1}
        self.bar = {(b, i): Bar(f"{b}{i}", count(b, fp8)) for b, n in sizes.items() for i in range(n)}
        self.tag, self.readers, self.landing, self.loads, self.tensor = {}, {}, set(), [], []
        self.info = {}
        self.s = [("free",), ("free",)]      # scores / weights of a warpgroup
        self.o = [None, None]                # (item, blocks summed)
        self.o_readers = [0, 0]

    def wait(self, b, i, need):
        """Until `need` phases are done, seen as the kernel sees them: by the parity of the last of them."""
        bar, parity = self.bar[b, i], (need - 1) & 1

        def ok():
            assert need - 1 <= bar.done <= need, f"{bar.name}: {bar.done} phases done, waiting for {need}"
            return (bar.done & 1) != parity
        return ok

    def arrive(self, b, i=0):
        self.bar[b, i].arrive()

    def use(self, buf, tag):
        assert buf not in self.landing, f"{buf} read while a copy lands"
        assert self.tag.get(buf) == tag, f"{buf} holds {self.tag.get(buf)}, expected {tag}"

    def hold(self, buf, by):
        self.readers[buf] = self.readers.get(buf, 0) + by

    def write(self, buf):
        assert not self.readers.get(buf), f"{buf} written while it is read"
        assert buf not in self.landing, f"two copies into {buf}"

    def load(self, buf, tag, b, i):
        self.write(buf)
        self.landing.add(buf)
        self.loads.append((buf, tag, b, i))

    # the order of a piece's tiles: K0 K1 V0 K2 V1 .. V(nb-2) V(nb-1)
    @staticmethod
    def tiles(nb):
        out = [("K", 0)]
        for b in range(1, nb):
            out += [("K", b), ("V", b - 1)]
        return out + [("V", nb - 1)]

    def producer(self):
        nq = nload = 0
        for n, (tok, nb) in enumerate(self.items + [(0, 0)]):
            yield self.wait("info_empty", n % INFO, n // INFO)
            self.info[n % INFO] = (tok, nb)
            self.arrive("info_full", n % INFO)
            for j, (kind, b) in enumerate(self.tiles(nb) if nb else []):
                ring, names = (self.R, ("raw", "raw_empty", "raw_full")) if self.fp8 else (self.T, ("kv", "kv_empty", "kv_full"))
                s = nload % ring
                yield self.wait(names[1], s, nload // ring)
                self.load((names[0], s), (n, kind, b), names[2], s)
                nload += 1
                if j == 0:
                    for q in range(2 if tok > 8 else 1):
                        yield self.wait("q_empty", nq % 2, nq // 2)
                        self.load(("q", nq % 2), (n, q), "q_full", nq % 2)
                        nq += 1

    def widen(self, w):
        base = nq = 0
        for n in range(len(self.items) + 1):
            yield self.wait("info_full", n % INFO, n // INFO + 1)
            tok, nb = self.info[n % INFO]
            self.arrive("info_empty", n % INFO)
            for j, (kind, b) in enumerate(self.tiles(nb) if nb else []):
                load = 2 * base + j
                r, t = load % self.R, load % self.T
                turns = load // (4 if self.mistake == "phase" else self.R)
                yield self.wait("raw_full", r, turns + 1)
                self.use(("raw", r), (n, kind, b))
                self.hold(("raw", r), 1)
                yield None
                self.hold(("raw", r), -1)
                self.arrive("raw_empty", r)
                yield self.wait("kv_empty", t, load // self.T)
                self.write(("kv", t))
                self.tag["kv", t] = (n, kind, b)
                yield None
                self.arrive("kv_full", t)
                for _ in range((2 if tok > 8 else 1) if j == 0 else 0):
                    yield self.wait("q_full", nq % 2, nq // 2 + 1)
                    yield None
                    self.arrive("q_ready", nq % 2)
                    nq += 1
            base += nb

    def mma(self):
        base = nq = 0
        pcount = [0, 0]
        for n in range(len(self.items) + 1):
            yield self.wait("info_full", n % INFO, n // INFO + 1)
            tok, nb = self.info[n % INFO]
            self.arrive("info_empty", n % INFO)
            if nb == 0:
                return
            dual = tok > 8
            order = {x: j for j, x in enumerate(self.tiles(nb))}

            def issue(w, bo, bs, base=base, nq=nq, n=n, nb=nb, dual=dual, order=order):
                first, last = not dual or w == 0, not dual or w == 1
                place = lambda kind, b: (2 * base + order[kind, b])  # noqa: E731
                if bo >= 0:
                    v = place("V", bo)
                    if first:
                        yield self.wait("kv_full", v % self.T, v // self.T + 1)
                    yield self.wait("p_full", w, pcount[w] + 1)
                    pcount[w] += 1
                    self.product(("O", w, n, bo), ("kv", v % self.T), (n, "V", bo))
                    if last:
                        self.tensor.append(("commit", "kv_empty", v % self.T))
                    if bs < 0:
                        self.tensor.append(("commit", "o_full", w))
                if bs >= 0:
                    k, qs = place("K", bs), (nq + w if dual else nq) % 2
                    if first:
                        yield self.wait("kv_full", k % self.T, k // self.T + 1)
                    self.product(("S", w, n, bs), ("kv", k % self.T), (n, "K", bs), ("q", qs), (n, w if dual else 0))
                    self.tensor.append(("commit", "s_full", w))
                    if first if self.mistake == "first reader" else last:
                        self.tensor.append(("commit", "kv_empty", k % self.T))
                    if bs == nb - 1:
                        self.tensor.append(("commit", "q_empty", qs))

            for t in range(nq, nq + (2 if dual else 1)):
                yield self.wait("q_ready" if self.fp8 else "q_full", t % 2, t // 2 + 1)
            steps = []
            if dual:
                steps = [(0, -1, 0), (1, -1, 0)]
                for b in range(nb):
                    steps += [(w, b, b + 1 if b + 1 < nb else -1) for w in (0, 1)]
            else:
                steps = [(0, -1, 0)] + ([(1, -1, 1)] if nb > 1 else [])
                steps += [(b % 2, b, b + 2 if b + 2 < nb else -1) for b in range(nb)]
            if self.mistake == "early scores" and len(steps) > 2:
                w, bo, bs = steps[2]
                if bs >= 0:
                    steps[2:3] = [(w, -1, bs), (w, bo, bs)]
            for step in steps:
                yield from issue(*step)
            base += nb
            nq += 2 if dual else 1

    def product(self, what, buf, tag, *q):
        # waited for: what it reads is there now, and stays until the product has executed
        self.use(buf, tag)
        held = [buf]
        if q:
            self.use(*q)
            held.append(q[0])
        for b in held:
            self.hold(b, 1)
        self.tensor.append((what[0], what[1:], held))

    def execute(self):
        kind, *rest = self.tensor.pop(0)
        if kind == "commit":
            self.arrive(*rest)
            return
        (w, n, b), held = rest
        if kind == "S":
            assert self.s[w][0] == "free", f"S of block {b} over {self.s[w]}"
            self.s[w] = ("S", n, b, 0)
        else:
            assert self.s[w] == ("P", n, b), f"O of item {n}, block {b}, from {self.s[w]}"
            self.s[w] = ("free",)
            if self.o[w] is None or self.o[w][0] != n:
                assert not self.o_readers[w], "O overwritten while it is read"
                assert self.o[w] is None or self.o[w][2] == 4, f"O of item {self.o[w][0]} overwritten unread"
                self.o[w] = (n, [], 0)
            self.o[w][1].append(b)
        for x in held:
            self.hold(x, -1)

    def softmax(self, warp):
        wg = warp // 4
        scount = ocount = xcount = 0
        for n in range(len(self.items) + 1):
            yield self.wait("info_full", n % INFO, n // INFO + 1)
            tok, nb = self.info[n % INFO]
            self.arrive("info_empty", n % INFO)
            if nb == 0:
                return
            dual = tok > 8
            mine = list(range(nb)) if dual else list(range(wg, nb, 2))
            for b in mine:
                yield self.wait("s_full", wg, scount + 1)
                scount += 1
                assert self.s[wg][:3] == ("S", n, b), f"scores {self.s[wg]}, expected block {b} of item {n}"
                yield None
                done = self.s[wg][3] + 1
                self.s[wg] = ("P", n, b) if done == 4 else ("S", n, b, done)
                yield None
                self.arrive("p_full", wg)
            if mine and self.mistake != "no order":
                yield self.wait("o_full", wg, ocount + 1)
                ocount += 1
            shared = not dual and nb > 1
            if shared:
                self.arrive("x_full")
                yield self.wait("x_full", 0, xcount + 1)
            for g in ((0, 1) if shared else (wg,) if mine else ()):
                want = list(range(nb)) if dual else list(range(g, nb, 2))
                assert self.o[g] and self.o[g][0] == n and self.o[g][1] == want, f"sums {self.o[g]} of item {n}, expected {want}"
                self.o_readers[g] += 1
            yield None
            for g in ((0, 1) if shared else (wg,) if mine else ()):
                self.o_readers[g] -= 1
                if g == wg:
                    self.o[g] = self.o[g][:2] + (self.o[g][2] + 1,)
            if shared:
                self.arrive("x_done")
                yield self.wait("x_done", 0, xcount + 1)
                xcount += 1

    def run(self):
        roles = [self.producer(), self.mma()] + [self.softmax(w) for w in range(8)] + [self.widen(w) for w in range(self.W)]
        blocked, live, steps = [None] * len(roles), set(range(len(roles))), 0
        while live or self.loads or self.tensor:
            steps += 1
            assert steps < 200000, "no progress"
            moves = [("role", r) for r in live if blocked[r] is None or blocked[r]()]
            moves += [("land", k) for k in range(len(self.loads))] + ([("tensor", 0)] if self.tensor else [])
            assert moves, "deadlock"
            kind, x = self.rng.choice(moves)
            if kind == "land":
                buf, tag, b, i = self.loads.pop(x)
                self.landing.discard(buf)
                self.tag[buf] = tag
                self.arrive(b, i)
            elif kind == "tensor":
                self.execute()
            else:
                try:
                    blocked[x] = next(roles[x])
                except StopIteration:
                    live.discard(x)


def pieces(rng, n):
    return [(rng.choice([1, 3, 8, 9, 16, 16]), rng.randint(1, 7)) for _ in range(n)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seed", range(12))
def test_random_schedules(seed, fp8):
    rng = random.Random(seed)
    Sim(pieces(rng, rng.randint(1, 12)), fp8, rng).run()


@pytest.mark.parametrize("fp8", [False, True])
def test_no_pieces_and_single_blocks(fp8):
    for items in ([], [(1, 1)], [(16, 1)] * 9, [(4, 1), (16, 2)] * 5):
        Sim(items, fp8, random.Random(len(items))).run()


@pytest.mark.parametrize("mistake,fp8", [("first reader", False), ("first reader", True), ("phase", True),
                                         ("early scores", False), ("no order", False)])
def test_planted_mistakes_are_reported(mistake, fp8):
    reported = 0
    for seed in range(20):
        rng = random.Random(seed)
        try:
            Sim(pieces(rng, 8), fp8, rng, mistake).run()
        except AssertionError:
            reported += 1
    assert reported >= 10, f"{mistake}: reported in {reported} of 20 runs"
