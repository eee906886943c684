"""Host models of the int8 cache's barriers in the chunk attention: those of the E4M3 cache, with six widening warps that take
no queries, and one-token items whose blocks lie in four places of which each belongs to the same four warps."""
import random
import re

import pytest

import test_chunk_attend_one_protocol as one
import test_chunk_attend_protocol as tile
from _kernel_consts import _source

TEXT = _source("chunk_attend.cu")
HELP = int(re.search(r"static constexpr int kHelp = kKv == kCaI8 \? (\d+) : 0;", TEXT).group(1))
PLACES = int(re.search(r"static constexpr int kOnePlaces = kKv == kCaI8 \? (\d+) : kCaOnePlaces;", TEXT).group(1))
LANES = int(re.search(r"lane < \(kI8 \? (\d+) : 1\)\) mbar_arrive\(&sm.one_empty", TEXT).group(1))


def _counts(barrier):
    """The arrival count behind `else mbar_init(..)`, where the int8 cache has one of its own."""
    e = re.search(r"else mbar_init\(&sm\." + barrier + r"\[i\], ([^)]+)\)", TEXT)
    return eval(e.group(1).replace("Shape::kHelp", str(HELP)).replace("Shape::kWiden", str(tile.shape("kWiden", True))))


class Tiles(tile.Sim):
    """No queries to widen: their arrivals come with the copies (the model's widening warps make them)."""

    def __init__(self, items, rng, mistake=None):
        super().__init__(items, True, rng, mistake)
        self.W += HELP
        for (b, i), bar in self.bar.items():
            n = self.W if b == "q_ready" else _counts(b) if b in ("kv_full", "raw_empty", "info_empty") else bar.n
            bar.n = bar.pending = n


@pytest.mark.parametrize("seed", range(12))
def test_tiles(seed):
    rng = random.Random(seed)
    Tiles(tile.pieces(rng, rng.randint(1, 12)), rng).run()


@pytest.mark.parametrize("mistake", ["first reader", "phase"])
def test_planted_mistakes_in_tiles_are_reported(mistake):
    reported = 0
    for seed in range(20):
        rng = random.Random(seed)
        try:
            Tiles(tile.pieces(rng, 8), rng, mistake).run()
        except AssertionError:
            reported += 1
    assert reported >= 10, f"{mistake}: reported in {reported} of 20 runs"


class OneTokens(one.Sim):
    def __init__(self, items, rng, mistake=None):
        super().__init__(items, True, rng, mistake)

    def release(self, s):
        self.unread[s] -= 2  # (counted in all eight warps' turns)
        for _ in range(LANES):
            self.arrive("one_empty", s)

    def attend(self, w):
        place = 0
        for n in range(len(self.items) + 1):
            yield self.wait("one_info_full", n % one.INFO, n // one.INFO + 1)
            item, nb = self.info[n % one.INFO]
            assert item == n
            self.arrive("one_info_empty", n % one.INFO)
            if nb == 0:
                return
            for b in range(nb):
                mine, s = (place & 1) == w >> 2, place % one.PLACES
                place += 1
                if not mine:
                    continue
                yield self.wait("one_full", s, (place - 1) // one.PLACES + 1)
                assert self.flag[s] == (n, b)
                if self.mistake == "early":
                    self.release(s)
                yield None
                self.use(s, (n, b, "KV"))
                if self.mistake != "early":
                    self.release(s)
            assert not self.readers[w]
            self.sums[w] = n
            yield None
            self.arrive("one_x_full")
            yield self.wait("one_x_full", 0, n + 1)
            for x in range(one.WARPS):
                assert self.sums[x] == n
                self.readers[x] += 1
            yield None
            for x in range(one.WARPS):
                self.readers[x] -= 1
            self.joined.append((n, w))
            self.arrive("one_x_done")
            yield self.wait("one_x_done", 0, n + 1)


@pytest.mark.parametrize("seed", range(12))
def test_one_token_items(seed, monkeypatch):
    monkeypatch.setattr(one, "PLACES", PLACES)
    assert PLACES % 2 == 0 and LANES * 4 == one.count("one_empty")
    rng = random.Random(seed)
    OneTokens([rng.randint(1, 9) for _ in range(rng.randint(0, 9))], rng).run()


def test_a_planted_mistake_in_one_token_items_is_reported(monkeypatch):
    monkeypatch.setattr(one, "PLACES", PLACES)
    reported = 0
    for seed in range(20):
        rng = random.Random(seed)
        try:
            OneTokens([rng.randint(1, 9) for _ in range(8)], rng, "early").run()
        except AssertionError:
            reported += 1
    assert reported >= 10
