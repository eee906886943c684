"""Attention over shared prefixes, and chunk attention over an int8 cache, against a 64-bit implementation that knows of no
sharing: each request attends to all its keys through its own row of the page table."""
import math

import pytest
import torch

import _int8kv as i8
import block_sparse_attention_08_gb300 as msa
from _serving import D, G, H, PAGE, attend, check_attend, ints, offsets, pages

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(D)
KINDS = ["bf16", "e4m3", "int8"]


class Batch:
    """groups: (shared tokens, [(own old tokens, new tokens) ..]) or (None, [(old, new) ..]) for requests in no group."""

    def __init__(self, groups, kind, seed=0, powers=True, spare_rows=0):
        gen = torch.Generator().manual_seed(seed)
        self.kind, self.lens, news, self.off, self.shared = kind, [], [], [0], []
        rows, at = [], 0
        for shared, requests in groups:
            common = 0 if shared is None else shared // PAGE
            first = list(range(at, at + common))
            at += common
            for old, new in requests:
                n = (shared or 0) + old + new
                own = pages(n) - common
                rows.append(first + list(range(at, at + own)))
                at += own
                self.lens.append(n)
                news.append(new)
            if shared is None and not self.shared:
                self.off[0] = len(rows)
            elif shared is None:  # a group that shares nothing
                self.shared.append(0)
                self.off.append(len(rows))
            else:
                self.shared.append(shared)
                self.off.append(len(rows))
        perm = torch.randperm(at + 1, generator=gen)
        width = max(1, max(map(len, rows)))
        self.table = torch.zeros(len(rows), width, dtype=torch.int32)
        for r, row in enumerate(rows):
            self.table[r, :len(row)] = perm[row]
        self.table = self.table.cuda()
        self.pool, self.news = at + 1, news
        self.cu = offsets(news)
        self.q = torch.randn(sum(news) + spare_rows, H, D, generator=gen).bfloat16().cuda()
        self.k_scale = self.v_scale = 1.0
        if kind == "int8":
            self.cache = i8.cache(self.pool, seed + 1, powers=powers) + i8.cache(self.pool, seed + 2, powers=powers)
            self.cache = (self.cache[0], self.cache[2], self.cache[1], self.cache[3])
            self.k, self.v = i8.values(self.cache[0], self.cache[2]), i8.values(self.cache[1], self.cache[3])
        else:
            self.cache = tuple(torch.randn(self.pool * PAGE, G, D, generator=gen).bfloat16().cuda() for _ in range(2))
            if kind == "e4m3":
                self.cache = tuple(c.to(torch.float8_e4m3fn) for c in self.cache)
                self.k_scale, self.v_scale = 0.5, 0.25
            self.k, self.v = self.cache
        self.call = {"bf16": msa.msa_attend_shared, "e4m3": msa.msa_attend_shared_fp8kv, "int8": msa.msa_attend_shared_int8kv}[kind]
        self.plain = {"bf16": msa.msa_attend_chunk, "e4m3": msa.msa_attend_chunk_fp8kv, "int8": msa.msa_attend_chunk_int8kv}[kind]

    def more(self, kw):
        return dict(kw, k_scale=self.k_scale, v_scale=self.v_scale) if self.kind == "e4m3" else kw

    def run(self, **kw):
        return self.call(self.q, *self.cache, ints(self.lens), self.table, self.cu, ints(self.off), ints(self.shared), **self.more(kw))

    def run_plain(self, **kw):
        return self.plain(self.q, *self.cache, ints(self.lens), self.table, self.cu, **self.more(kw))

    def want(self, **kw):
        return attend(self.q, self.k, self.v, self.lens, self.table, self.cu, SCALE, self.k_scale, self.v_scale, **kw)

    def check(self, out, lse, ref, bits=None):
        check_attend(out, lse, ref, max(self.lens), bits or {"bf16": 8, "e4m3": 11, "int8": 8}[self.kind])


SHAPES = {
    "two, one page": [(128, [(0, 1), (5, 1)])],
    "a page and a bit": [(200, [(0, 1), (1, 1), (127, 1), (128, 1)])],
    "16 tokens": [(1000, [(i, 1) for i in range(16)])],
    "17 tokens": [(1000, [(i, 1) for i in range(17)])],
    "9 tokens, long": [(20011, [(7 * i, 1) for i in range(9)])],
    "100 requests": [(3000, [(13 * i, 1) for i in range(100)])],
    "drafted tokens": [(700, [(300 + i, 1 + i % 5) for i in range(23)])],
    "chunks and single tokens": [(2500, [(100, 1), (0, 40), (30, 1), (9, 17), (500, 1), (1, 12)])],
    "groups and others": [(None, [(0, 1), (900, 33)]), (400, [(50, 1), (60, 1)]), (None, [(300, 1)]), (1281, [(0, 2), (10, 1), (3, 1)]),
                          (128, [(1, 1)]), (None, [(2000, 5), (3, 1)])],
    "requests without new tokens": [(900, [(0, 0), (5, 1), (6, 0), (7, 2), (0, 0)])],
    "a group without tokens": [(900, [(10, 0), (5, 0)]), (300, [(5, 1), (8, 1)])],
    "more tokens than fill the items": [(600, [(0, 20), (3, 50)])],
    "48 groups": [(128 + 3 * g, [(g, 1)] * (2 + 7 * (g % 2))) for g in range(48)],
    "49 groups and others": [(256, [(g + i, 1) for i in range(2 + g % 9)]) for g in range(49)] + [(None, [(40, 1), (600, 3)])],
    "700 requests": [(256, [(i % 90, 1) for i in range(350)]), (384, [(i % 70, 1) for i in range(350)])],
}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", SHAPES)
def test_shared(name, kind):
    b = Batch(SHAPES[name], kind)
    lse = torch.empty(b.q.shape[:2], dtype=torch.float32, device="cuda")
    ws = msa.Workspace(msa.workspace_size(msa.make_config(), 5, b.q.shape[0], b.table.shape[1]))
    out = b.run(lse=lse, workspace=ws)
    assert ws.read_device_error() == (0, 0)
    b.check(out, lse, b.want())
    again = torch.empty_like(lse)
    assert torch.equal(out, b.run(lse=again)) and torch.equal(lse, again)


@pytest.mark.parametrize("powers", [True, False])
@pytest.mark.parametrize("requests", [
    [(0, 1)], [(0, 128), (1, 128), (127, 1)], [(300, 1), (0, 1), (5000, 1), (128, 1)], [(16000, 1)], [(0, 5), (700, 8), (90, 9)],
    [(3000, 500), (0, 333), (77, 16)], [(10 * i, 1 + i % 3) for i in range(60)]])
def test_chunk_int8(requests, powers):
    b = Batch([(None, requests)], "int8", powers=powers)
    lse = torch.empty(b.q.shape[:2], dtype=torch.float32, device="cuda")
    ws = msa.Workspace(msa.workspace_size(msa.make_config(), 4, b.q.shape[0], b.table.shape[1]))
    out = b.run_plain(lse=lse, workspace=ws)
    assert ws.read_device_error() == (0, 0)
    ref = b.want()
    if powers:
        b.check(out, lse, ref)
    else:
        # K and V may be rounded to bf16, by 2^-8 each: a score moves by up to 2^-8 of reach, as if its fp32 sum were off by that
        # much, and a value by 2^-8 of itself, as its weight's rounding would
        out_ref, lse_ref, spread, reach = ref
        score = 2.0 ** -8 * reach
        tol = 2.0 ** -8 * out_ref.abs() + 1.1 * (2 * score + 3 * 2.0 ** -8)[..., None] * spread + 2.0 ** -20
        assert bool(((out.double() - out_ref).abs() <= tol).all())
        assert bool(((lse.double() - lse_ref).abs() <= 1.4427 * 1.01 * score + 1e-4).all())


def test_no_groups_is_the_chunk_attention():
    for kind in KINDS:
        b = Batch([(None, [(500, 1), (3, 7), (0, 200)])], kind)
        b.off, b.shared = [0], []
        assert torch.equal(b.run(), b.run_plain())


@pytest.mark.parametrize("kind", KINDS)
def test_rows_behind_the_last_token_are_left(kind):
    b = Batch(SHAPES["drafted tokens"], kind, spare_rows=37)
    out = torch.full_like(b.q, 3.0)
    lse = torch.full(b.q.shape[:2], 3.0, device="cuda")
    b.run(out=out, lse=lse)
    t = sum(b.news)
    assert bool((out[t:] == 3).all()) and bool((lse[t:] == 3).all())
    ref = b.want()
    b.check(out[:t], lse[:t], tuple(x[:t] for x in ref))


@pytest.mark.parametrize("kind", KINDS)
def test_what_lies_behind_the_last_key_does_not_matter(kind):
    b = Batch(SHAPES["groups and others"], kind)
    ref = b.want()
    used = torch.zeros(b.pool * PAGE, dtype=torch.bool, device="cuda")
    for r, n in enumerate(b.lens):
        pos = torch.arange(n, device="cuda")
        used[b.table[r].long()[pos // PAGE] * PAGE + pos % PAGE] = True
    if kind == "int8":
        free = torch.nonzero(~used).flatten()
        for s in b.cache[2:]:
            s[free // PAGE, :, free % PAGE] = math.nan
    elif kind == "bf16":
        for c in b.cache:
            c[~used] = math.nan
    else:
        for c in b.cache:
            c.view(torch.uint8)[~used] = 0x7F
    lse = torch.empty(b.q.shape[:2], dtype=torch.float32, device="cuda")
    b.check(b.run(lse=lse), lse, ref)
    lse = torch.empty(b.q.shape[:2], dtype=torch.float32, device="cuda")
    b.check(b.run_plain(lse=lse), lse, ref)


@pytest.mark.parametrize("kind", KINDS)
def test_bad_lengths_and_pages(kind):
    b = Batch([(600, [(100, 1), (100, 2), (100, 1)] + [(20, 2)] * 3), (300, [(5, 5), (6, 5)])], kind)
    ws = msa.Workspace(msa.workspace_size(msa.make_config(), 5, b.q.shape[0], b.table.shape[1]))
    ref = b.want()
    lens = list(b.lens)
    b.lens[1] = 500                               # fewer tokens than its group shares
    lse = torch.empty(b.q.shape[:2], dtype=torch.float32, device="cuda")
    out = b.run(lse=lse, workspace=ws)
    assert ws.read_device_error() == (3, 1)
    assert bool((out[1:3] == 0).all()) and bool((lse[1:3] == -math.inf).all())
    good = [0] + list(range(3, len(out)))
    b.check(out[good], lse[good], tuple(x[good] for x in ref))
    b.lens = lens
    table = b.table.clone()
    for page in (-1, b.pool):
        b.table[0, 2] = page                      # a shared page: its keys are missing for the whole group
        out = b.run(lse=lse, workspace=ws)
        assert ws.read_device_error() == (1, 2)
        b.check(out, lse, b.want(skip=[(r, 2) for r in range(6)]))
        b.table.copy_(table)
        b.table[7, 2] = page                      # one of a request's own
        out = b.run(lse=lse, workspace=ws)
        assert ws.read_device_error() == (1, 7 * table.shape[1] + 2)
        b.check(out, lse, b.want(skip=[(7, 2)]))
        b.table.copy_(table)


def test_small_groups_have_the_same_lengths_to_keep():
    """A group whose pages are read for each request (few tokens) refuses the requests that the others would."""
    for requests in ([(100, 1), (50, 1), (60, 1)], [(10, 1)], [(10, 40), (20, 50)]):
        b = Batch([(600, requests)], "bf16")
        ws = msa.Workspace(msa.workspace_size(msa.make_config(), 5, b.q.shape[0], b.table.shape[1]))
        ref = b.want()
        b.check(b.run(workspace=ws), None, ref)
        assert ws.read_device_error() == (0, 0)
        b.lens[0] = 512 + requests[0][1] - 1      # 511 tokens before the new ones, four whole pages are shared
        out = b.run(workspace=ws)
        assert ws.read_device_error() == (3, 0)
        n = requests[0][1]
        assert bool((out[:n] == 0).all())
        if len(requests) > 1:
            b.check(out[n:], None, tuple(x[n:] for x in ref))


@pytest.mark.parametrize("off,shared", [([-1, 3], [256]), ([1, 9], [256]), ([4, 2], [256]), ([3, 4], [256]), ([0, 5], [-7]),
                                        ([0, 0, 0, 5], [256, 256, 0]), ([5, 5], [128])])
def test_groups_that_share_nothing(off, shared):
    b = Batch([(None, [(600, 1), (300, 3), (5, 1), (700, 1), (900, 2)])], "bf16")
    b.off, b.shared = off, shared
    b.check(b.run(), None, b.want())


def test_a_key_that_is_not_finite_reaches_its_own_rows_alone():
    b = Batch([(256, [(40, 1), (50, 1), (60, 1)])], "int8")
    clean = b.run()
    slot = int(b.table[1, 2]) * PAGE + 3          # a key of the second request, and one of its values
    for s in b.cache[2:]:
        s[slot // PAGE, 2, slot % PAGE] = math.nan
    out = b.run()
    assert bool(out[1, 32:48].isnan().all())
    rest = torch.ones(3, H, dtype=torch.bool, device="cuda")
    rest[1, 32:48] = False
    assert torch.equal(out[rest], clean[rest])


def test_calls_on_two_streams_and_a_replayed_graph():
    batches = [Batch(SHAPES["100 requests"], k, seed=i) for i, k in enumerate(KINDS)]
    want = [b.run() for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    args = [(ints(b.lens), ints(b.off), ints(b.shared)) for b in batches]
    torch.cuda.synchronize()
    got = [[], [], []]
    for _ in range(10):
        for b, s, g, (lens, off, shared) in zip(batches, streams, got, args):
            with torch.cuda.stream(s):
                g.append(b.call(b.q, *b.cache, lens, b.table, b.cu, off, shared, **b.more({})))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)
    b, (lens, off, shared) = batches[2], args[2]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.call(b.q, *b.cache, lens, b.table, b.cu, off, shared)
    for less in (0, 7):
        lens.copy_(ints([n - less if n - less > b.shared[0] else n for n in b.lens]))
        out.fill_(9)
        graph.replay()
        expect = b.call(b.q, *b.cache, lens, b.table, b.cu, off, shared)
        assert torch.equal(out, expect)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name,plain", [("16 tokens", False), ("9 tokens, long", False), ("drafted tokens", False), ("chunks and single tokens", True),
                                        ("drafted tokens", True)])
def test_calls_behind_one_another_give_the_same_bits(name, plain, kind):
    """Many calls with nothing between them: a tile that is given back before it has been read shows in some of them."""
    b = Batch(SHAPES[name], kind)
    lens, off, shared = ints(b.lens), ints(b.off), ints(b.shared)
    args = (b.q, *b.cache, lens, b.table, b.cu) + (() if plain else (off, shared))
    call = b.plain if plain else b.call
    outs = [call(*args, **b.more({})) for _ in range(60)]
    assert all(torch.equal(outs[0], x) for x in outs)


def _poison(b, name, slot, g):
    """A key ("k") or a value ("v") that is not finite."""
    i = "kv".index(name)
    if b.kind == "int8":
        b.cache[2 + i][slot // PAGE, g, slot % PAGE] = math.nan
    elif b.kind == "bf16":
        b.cache[i][slot, g, 5] = math.nan
    else:
        b.cache[i].view(torch.uint8)[slot, g, 5] = 0x7F


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("where", ["query", "only own key", "only own value", "shared key", "one of the own keys"])
@pytest.mark.parametrize("tokens", [9, 20, 60])
def test_what_is_not_finite_stays_so_where_pieces_are_joined(tokens, where, kind):
    """Requests that bring one token each (every third one two) behind a whole number of shared pages; a group's items are cut
    into pieces for few tokens and for many.  As in the chunk attention, what a number is missing for is NaN, and
    nothing else changes."""
    b = Batch([(20 * PAGE, [(0 if i % 2 else 200, 2 if i % 3 == 2 else 1) for i in range(tokens)])], kind)
    r, g = 7, 2                                    # (a request with one new token and no other own key)
    t, heads = sum(b.news[:r]), slice(16 * g, 16 * g + 16)
    lse = torch.empty(b.q.shape[:2], dtype=torch.float32, device="cuda")
    clean = b.run(lse=lse)
    clean_lse = lse.clone()
    bad = torch.zeros(b.q.shape[:2], dtype=torch.bool, device="cuda")
    if where == "query":
        b.q[t, 16 * g + 3] = math.nan
        bad[t, 16 * g + 3] = True
    elif where == "shared key":
        _poison(b, "k", int(b.table[0, 3]) * PAGE + 17, g)
        bad[:, heads] = True
    elif where == "one of the own keys":           # its only page: 201 keys
        r, t = 6, sum(b.news[:6])
        _poison(b, "k", int(b.table[r, 20]) * PAGE + 40, g)
        bad[t:t + b.news[r], heads] = True
    else:
        _poison(b, "k" if where == "only own key" else "v", int(b.table[r, 20]) * PAGE, g)
        bad[t, heads] = True
    assert b.news[7] == 1 and b.lens[7] == 20 * PAGE + 1
    plain_lse = torch.empty_like(lse)
    plain = b.run_plain(lse=plain_lse)
    out = b.run(lse=lse)
    nan = out.isnan()
    assert torch.equal(nan.all(-1), bad) or where == "only own value"
    assert torch.equal(nan, plain.isnan()) and torch.equal(lse.isnan(), plain_lse.isnan())
    assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad])
    if where != "only own value":
        assert torch.equal(lse.isnan(), bad)
