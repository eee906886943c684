"""Host model of how the shared-prefix attention shares out its work (chunk_attend.cu with kShared: ca_find_shares, the walks of
the producer warp, CaPieces and shared_join_kernel).

Random batches of groups and requests are cut into the CTAs' shares as the kernel cuts them.  Every (token, KV head, block) has to
be attended to exactly once, no two pieces may leave their sums in the same place, and the pieces that the join reads for a token
have to be those that hold its sums.  Planted mistakes have to be found.  No GPU is involved.
"""
import random

import pytest

from _kernel_consts import kconst

FILE = "chunk_attend.cu"
TOK, CTAS = kconst("kCaTok", FILE), kconst("kNumSMs", FILE)
BLOCK = 128


def eighths(x):
    q = x >> 3
    return 4 * q * (q - 1) + q * (x & 7)


class Entry:
    def __init__(self, t0=0, n=0, length=0, skip=0, whole=False):
        self.t0, self.n, self.len, self.skip, self.whole, self.extra, self.extra1 = t0, n, length, skip, whole, 0, 0

    def one(self):
        return not self.whole and self.n % TOK == 1

    def items(self):
        return (self.n + TOK - 1) // TOK - self.one()

    def blocks(self, i):
        if self.whole:
            return self.len // BLOCK
        return (self.len - self.n + min(self.n, TOK * (i + 1)) - 1) // BLOCK + 1 - self.skip

    def dual(self, i):
        return self.n - TOK * i > TOK // 2

    def before(self, i):
        if self.whole:
            return (self.len // BLOCK + self.extra) * i
        a = (self.len - self.n + TOK - 1) // TOK
        return eighths(a + i) - eighths(a) + i + (self.extra - self.skip) * i

    def units(self, i):
        return self.extra + (self.blocks(i) if self.dual(i) else (self.blocks(i) + 1) // 2)

    def per_head(self):
        i = self.items() - 1
        return 0 if i < 0 else self.before(i) + self.units(i)

    def one_blocks(self):
        return (self.len - 1) // BLOCK + 1 - self.skip

    def one_units(self):
        return (self.one_blocks() + 1) // 2 + self.extra1 if self.one() else 0

    def one_begun(self, x):
        return min(self.one_blocks(), 0 if x <= 0 else 2 * (1 + max(0, x - 1 - self.extra1)))

    def joined(self):
        return self.whole or self.skip > 0


def group(g, offsets, shared, cu, batch, tokens, max_blocks):
    r0, r1, blocks = offsets[g], offsets[g + 1], int(shared[g] / BLOCK)
    if r0 < 0 or r1 > batch or r1 <= r0 or r1 - r0 < 2 or blocks < 1:
        return r0, r1, 0, 0, 0
    c0, c1 = cu[r0], cu[r1]
    if c0 < 0 or c1 < c0 or c1 > tokens or c1 - c0 >= TOK * (r1 - r0):
        return r0, r1, 0, 0, 0
    return r0, r1, min(blocks, max_blocks), c0, c1 - c0


def entries(lens, cu, offsets, shared, tokens, max_blocks, bad):
    batch, groups, out = len(lens), len(shared), []
    for g in range(groups):
        r0, r1, blocks, t0, n = group(g, offsets, shared, cu, batch, tokens, max_blocks)
        out.append(Entry(t0, n, blocks * BLOCK, 0, True) if blocks else Entry())
    for r in range(batch):
        lo, hi = 0, groups
        while lo < hi:
            mid = lo + (hi - lo) // 2
            if offsets[mid + 1] > r:
                hi = mid
            else:
                lo = mid + 1
        skip = 0
        if lo < groups:
            r0, _, blocks, _, _ = group(lo, offsets, shared, cu, batch, tokens, max_blocks)
            skip = blocks if r0 <= r else 0
        c0, c1 = cu[r], cu[r + 1]
        good = 0 <= c0 <= c1 <= tokens and c1 - c0 <= lens[r] and -(-lens[r] // BLOCK) <= max_blocks
        if good and (c0 == c1 or lens[r] - (c1 - c0) >= skip * BLOCK):
            out.append(Entry(c0, c1 - c0, lens[r], skip))
        else:
            bad.update(range(max(0, c0), min(tokens, c1)))
            out.append(Entry())
    return out


def split(total, c, extra):
    ctas = min(CTAS, max(total // (1 + extra), 1))
    return ctas, min(total, total * c // ctas), min(total, total * (c + 1) // ctas)


def walk(work, c, extra, total, emit, mistake):
    """The items of two and more tokens of CTA c."""
    ctas, u0, u1 = split(total, c, extra)
    if u0 >= u1:
        return
    base = 0
    for e, q in enumerate(work):
        if base <= u0 < base + 4 * q.per_head():
            break
        base += 4 * q.per_head()
    per = q.per_head()
    g, rem = (u0 - base) // per, (u0 - base) % per
    i = max(j for j in range(q.items()) if q.before(j) <= rem)
    at, item0 = u0, u0 - (rem - q.before(i))
    while True:
        blocks, dual, end = q.blocks(i), q.dual(i), item0 + q.units(i)

        def begun(x):
            units = 0 if x <= 0 else 1 + max(0, x - 1 - q.extra)
            return min(blocks, units if dual else 2 * units)
        b0 = begun(at - item0)
        nb = begun(min(end, u1) - item0) - b0
        to_end = b0 + nb == blocks
        if nb > 0:
            t0, ntok = q.t0 + TOK * i, min(TOK, q.n - TOK * i)
            slot = ("token", q.whole) if b0 == 0 and to_end and q.joined() else ("out",) if b0 == 0 and to_end else ("cta", 2 * c + (b0 == 0))
            last = (end * ctas - 1) // total
            if mistake == "last":
                last = (end * ctas) // total
            emit(q, t0, ntok, g, b0 + q.skip, nb, slot, False, b0 == 0 and (not to_end, last), c)
        at = item0 = end
        if at >= u1:
            return
        i += 1
        if i == q.items():
            i, g = 0, g + 1
            if g == 4:
                g = 0
                while True:
                    e += 1
                    q = work[e]
                    if q.items() > 0:
                        break


def walk_one(work, cta, extra1, total, emit, mistake):
    c = CTAS - 1 - cta
    ctas, u0, u1 = split(total, c, extra1)
    if u0 >= u1:
        return
    base = 0
    for e, q in enumerate(work):
        if base <= u0 < base + 4 * q.one_units():
            break
        base += 4 * q.one_units()
    per = q.one_units()
    g, u, at = (u0 - base) // per, (u0 - base) % per, u0
    while True:
        to = min(per, u + u1 - at)
        nb = q.one_begun(to) - q.one_begun(u)
        begins, whole = u == 0, u == 0 and nb == q.one_blocks()
        slot = ("token", False) if whole and q.joined() else ("out",) if whole else ("one", 2 * c + begins)
        skip = 0 if mistake == "skip" else q.skip
        if nb > 0:
            emit(q, q.t0 + q.n - 1, 1, g, q.one_begun(u) + skip, nb, slot, True,
                 begins and (not whole, ((at + per) * ctas - 1) // total), c)
        at += to - u
        if at >= u1:
            return
        u, g = 0, g + 1
        if g == 4:
            g = 0
            while True:
                e += 1
                q, per = work[e], work[e].one_units()
                if per:
                    break


def check(lens, news, offsets, shared, mistake=None):
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    tokens, max_blocks, bad = cu[-1], max(-(-n // BLOCK) for n in lens), set()
    work = entries(lens, cu, offsets, shared, tokens, max_blocks, bad)
    total = 4 * sum(q.per_head() for q in work)
    extra = 2 if total >= 16 * CTAS else 1 if total >= 4 * CTAS else 0
    ones = 4 * sum(q.one_units() for q in work)
    extra1 = 1 if ones >= 4 * CTAS else 0
    for q in work:
        q.extra, q.extra1 = extra, extra1
    total = 4 * sum(q.per_head() for q in work)
    ones = 4 * sum(q.one_units() for q in work)
    seen, places, own, with_, direct = {}, {}, {}, {}, {}

    def emit(q, t0, ntok, g, b0, nb, slot, one, begin, c):
        assert nb > 0 and ntok > 0
        for e in range(ntok):
            for b in range(b0, b0 + nb):
                key = (t0 + e, g, b)
                assert key not in seen, f"{key} twice"
                seen[key] = True
            if slot[0] == "out":
                direct[t0 + e, g] = nb
            else:
                place = ("token", slot[1], t0 + e, g) if slot[0] == "token" else (*slot, e)
                assert place not in places, f"{place} twice"
                places[place] = (t0 + e, g, q.whole, b0, nb)
            if begin:
                at = with_ if q.whole else own
                assert (t0 + e, g) not in at
                at[t0 + e, g] = (begin[0] or q.joined(), q.joined(), begin[0], one, c, begin[1], e)
    for c in range(CTAS):
        walk(work, c, extra, total, emit, mistake)
        walk_one(work, c, extra1, ones, emit, mistake)
    # each good token's keys, once; each of its pieces where the join looks for it
    request = [r for r, n in enumerate(news) for _ in range(n)]
    read = set()
    for t in range(tokens):
        r = request[t]
        if t in bad:
            continue
        blocks = (lens[r] - news[r] + (t - cu[r]) // TOK * TOK + min(TOK, news[r] - (t - cu[r]) // TOK * TOK) - 1) // BLOCK + 1
        for g in range(4):
            assert all((t, g, b) in seen for b in range(blocks)), (t, g)
            join, part, cut, one, first, last, e = own[t, g]
            if not join:
                assert direct[t, g] == blocks
                continue
            held = 0
            for whole, (_, _, cut, one, first, last, e) in [(False, own[t, g])] + ([(True, with_[t, g])] if part else []):
                if cut:
                    assert 0 <= first <= last < CTAS
                    for s in range(last - first + 1):
                        place = ("one" if one else "cta", 2 * first + 1 if s == 0 else 2 * (first + s), e)
                        assert place in places and places[place][:3] == (t, g, whole), (place, places.get(place))
                        held += places[place][4]
                        read.add(place)
                else:
                    place = ("token", whole, t, g)
                    assert places[place][:3] == (t, g, whole)
                    held += places[place][4]
                    read.add(place)
            assert held == blocks
    # (what a group computed for a request with bad lengths is not read)
    assert all(p in read or places[p][0] in bad for p in places)


def batch(rng):
    lens, news, offsets, shared = [], [], [], []
    for _ in range(rng.choice([1, 1, 2, 5])):
        for _ in range(rng.choice([0, 0, 3])):  # requests that share nothing
            news.append(rng.choice([0, 1, 1, 17, 40]))
            lens.append(news[-1] + rng.randint(0, 3000))
        if not offsets:
            offsets.append(len(lens))
        shared.append(rng.choice([100, 128, 1000, 20000, 65536]))
        most = rng.choice([1, 1, 4, 15, 40])
        for _ in range(rng.choice([0, 1, 2, 3, 40, 200])):
            news.append(rng.randint(0 if rng.random() < 0.2 else 1, most))
            old = shared[-1] + rng.choice([0, rng.randint(0, 40), rng.randint(0, 3000)])
            if rng.random() < 0.03:
                old = rng.randint(0, shared[-1])  # (perhaps too few)
            lens.append(old + news[-1])
        offsets.append(len(lens))
    if not lens:
        return batch(rng)
    if not sum(news):
        news[0] += 1
        lens[0] += 1
    return [max(n, 1) for n in lens], news, offsets, shared


@pytest.mark.parametrize("seed", range(60))
def test_every_key_once_and_every_piece_found(seed):
    check(*batch(random.Random(seed)))


@pytest.mark.parametrize("mistake", ["last", "skip"])
def test_planted_mistakes_are_found(mistake):
    found = 0
    for seed in range(20):
        try:
            check(*batch(random.Random(seed)), mistake)
        except (AssertionError, KeyError):
            found += 1
    assert found >= 5


@pytest.mark.parametrize("offsets,shared", [([-1, 3], [256]), ([2, 9], [256]), ([4, 2], [256]), ([2, 2], [256]), ([0, 1], [256]),
                                            ([0, 6], [0]), ([0, 6], [-500]), ([0, 6], [127]), ([0, 6], [599]), ([0, 6], [600])])
def test_odd_groups(offsets, shared):
    """Offsets that are no range, a single request, nothing shared, and as much as there is or more."""
    check([600] * 6, [1] * 6, offsets, shared)
