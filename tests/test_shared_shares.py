"""Host model of how the shared-prefix attention shares out its work (chunk_attend.cu with kShared: ca_find_shares, the walks of
the producer warp, CaPieces and shared_join_kernel).

Random batches of groups and requests are cut into the CTAs' shares as the kernel cuts them.  Every (token, KV head, block) has to
be attended to exactly once, no two pieces may leave their sums in the same place, and the pieces that the join reads for a token
have to be those that hold its sums.  Planted mistakes have to be found.  No GPU is involved.
"""
import random
import re

import pytest

from _kernel_consts import _source, kconst

FILE = "chunk_attend.cu"
FEW_TOKENS = kconst("kCaFewTokens", FILE)
FEW_BLOCKS = int(re.search(r"kCaFewBlocks = (\d+);", _source(FILE))[1])
TOK, CTAS = kconst("kCaTok", FILE), kconst("kNumSMs", FILE)
BLOCK = 128
_w = re.search(r"tile = kFp8 \|\| extra == 0 \? 1 : (\d+), token = kFp8 \|\| extra == 0 \? 1 : far \? (\d+) : (\d+);", _source(FILE))
WEIGHTS = {True: (int(_w[1]), int(_w[2])), False: (int(_w[1]), int(_w[3]))}  # of a unit of either kind, in long and short shares
FAR = int(re.search(r"far = total\[0\] \+ total\[2\] >= (\d+)LL", _source(FILE))[1])


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
    """(first request, blocks that its requests share, blocks attended to once, first token, tokens)."""
    r0, r1, blocks = offsets[g], offsets[g + 1], int(shared[g] / BLOCK)
    if r0 < 0 or r1 > batch or r1 <= r0 or blocks < 1:
        return r0, 0, 0, 0, 0
    some, c0, c1 = min(blocks, max_blocks), cu[r0], cu[r1]
    n = c1 - c0
    if c0 < 0 or n < 3 or c1 > tokens or r1 - r0 < 2 or n >= TOK * (r1 - r0) or (n < FEW_TOKENS and (n - 1) * some < FEW_BLOCKS):
        return r0, some, 0, 0, 0
    return r0, some, some, c0, n


def entries(lens, cu, offsets, shared, tokens, max_blocks, bad):
    batch, groups, out = len(lens), len(shared), []
    for g in range(groups):
        _, _, once, t0, n = group(g, offsets, shared, cu, batch, tokens, max_blocks)
        out.append(Entry(t0, n, once * BLOCK, 0, True) if once else Entry())
    for r in range(batch):
        lo, hi = 0, groups
        while lo < hi:
            mid = lo + (hi - lo) // 2
            if offsets[mid + 1] > r:
                hi = mid
            else:
                lo = mid + 1
        blocks = skip = 0
        if lo < groups:
            r0, blocks, skip, _, _ = group(lo, offsets, shared, cu, batch, tokens, max_blocks)
            if r0 > r:
                blocks = skip = 0
        c0, c1 = cu[r], cu[r + 1]
        good = 0 <= c0 <= c1 <= tokens and c1 - c0 <= lens[r] and -(-lens[r] // BLOCK) <= max_blocks
        if good and (c0 == c1 or lens[r] - (c1 - c0) >= blocks * BLOCK):
            out.append(Entry(c0, c1 - c0, lens[r], skip))
        else:
            bad.update(range(max(0, c0), min(tokens, c1)))
            out.append(Entry())
    return out


def split(n0, n1, c, extra, fp8, far):
    """For the tiles' items and for the one-token items: (units from .. to, what all shares are parts of, CTAs, before, weight)."""
    if fp8 and extra == 2:  # each kind by itself
        out = []
        for n, e in ((n0, extra), (n1, min(extra, 1))):
            ctas = min(CTAS, max(n // (1 + e), 1))
            out.append((min(n, n * c // ctas), min(n, n * (c + 1) // ctas), n, ctas, 0, 1))
        return out
    tile, token = (1, 1) if fp8 or extra == 0 else WEIGHTS[far]
    total = tile * n0 + token * n1
    ctas = min(CTAS, max(total // token // (1 + extra), 1))
    p0, p1 = total * min(c, ctas) // ctas, total * min(c + 1, ctas) // ctas
    return [(min(p0 // tile, n0), min(p1 // tile, n0), total, ctas, 0, tile),
            (max(p0 - tile * n0, 0) // token, max(p1 - tile * n0, 0) // token, total, ctas, tile * n0, token)]


def walk(work, c, share, emit, mistake):
    """The items of two and more tokens of CTA c."""
    u0, u1, total, ctas, before, weight = share
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
            last = ((before + weight * end) * ctas - 1) // total
            if mistake == "last":
                last = ((before + weight * (end - 1)) * ctas - 1) // total
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


def walk_one(work, c, share, emit, mistake):
    u0, u1, total, ctas, before, weight = share
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
                 begins and (not whole, ((before + weight * (at + per)) * ctas - 1) // total), c)
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


def check(lens, news, offsets, shared, mistake=None, fp8=False):
    cu = [0]
    for n in news:
        cu.append(cu[-1] + n)
    tokens, max_blocks, bad = cu[-1], max(-(-n // BLOCK) for n in lens), set()
    work = entries(lens, cu, offsets, shared, tokens, max_blocks, bad)
    both = 4 * sum(q.per_head() + q.one_units() for q in work)
    extra = 2 if both >= 16 * CTAS else 1 if both >= 4 * CTAS else 0
    for q in work:
        q.extra, q.extra1 = extra, min(extra, 1)
    n0, n1 = 4 * sum(q.per_head() for q in work), 4 * sum(q.one_units() for q in work)
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
        shares = split(n0, n1, c, extra, fp8, both >= FAR * CTAS)
        walk(work, c, shares[0], emit, mistake)
        walk_one(work, c, shares[1], emit, mistake)
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
    check(*batch(random.Random(seed)), fp8=seed % 2 == 1)


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
                                            ([0, 6], [0]), ([0, 6], [-500]), ([0, 6], [127]), ([0, 6], [599]), ([0, 6], [600]),
                                            ([0, 6], [639]), ([0, 6], [640]), ([0, 6], [2 ** 31 - 1])])
@pytest.mark.parametrize("each", [1, 2])
def test_odd_groups(offsets, shared, each):
    """Offsets that are no range, a single request, nothing shared, and as much as there is or more."""
    check([640] * 6, [each] * 6, offsets, shared)
