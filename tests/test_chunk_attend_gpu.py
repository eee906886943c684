"""Attention of a chunk of new tokens over the paged cache against a 64-bit implementation (the tolerance's
derivation stands in _serving.check_attend)."""
import math

import pytest
import torch

import _serving as S
import block_sparse_attention_08_gb300 as msa

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(128.0)
FP8 = {"bf16": False, "e4m3": True}


class Batch:
    def __init__(self, lens, news, cache="bf16", seed=0, width=None, rows=None, k_scale=0.5, v_scale=0.25, k_size=1.0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.lens, self.news, self.fp8 = lens, news, FP8[cache]
        self.table, pool = S.page_table(lens, width=width, spare=2, seed=seed)
        self.cu, self.seq = S.offsets(news), S.ints(lens)
        tokens = sum(news) if rows is None else rows
        self.q = torch.randn(tokens, 64, 128, generator=gen, device="cuda").bfloat16()
        kv = [torch.randn(pool * 128, 4, 128, generator=gen, device="cuda") * s for s in (k_size, 1.0)]
        self.k, self.v = (x.to(torch.float8_e4m3fn if self.fp8 else torch.bfloat16) for x in kv)
        self.scales = {"k_scale": k_scale, "v_scale": v_scale} if self.fp8 else {}

    def poison(self):
        """NaN and infinities wherever no request has a key."""
        used = torch.zeros(self.k.shape[0], dtype=torch.bool, device="cuda")
        for r, n in enumerate(self.lens):
            pos = torch.arange(n, device="cuda")
            used[self.table[r].long()[pos // 128] * 128 + pos % 128] = True
        for x in (self.k, self.v):
            if self.fp8:
                x.view(torch.uint8)[~used] = 0x7F  # E4M3's NaN
            else:
                x[~used] = math.nan
        if not self.fp8:
            self.v[~used, :, ::2] = math.inf
        return self

    def call(self, scale=SCALE, lse=True, **kw):
        f = msa.msa_attend_chunk_fp8kv if self.fp8 else msa.msa_attend_chunk
        out_lse = torch.full(self.q.shape[:2], 123.0, device="cuda") if lse else None
        out = kw.pop("out", None)
        out = torch.full_like(self.q, 77.0) if out is None else out
        got = f(self.q, self.k, self.v, self.seq, self.table, self.cu, scale=scale, out=out, lse=out_lse, **self.scales,
                **kw)
        assert got is out
        return got, out_lse

    def check(self, scale=SCALE, skip=(), **kw):
        got, lse = self.call(scale, **kw)
        n = sum(self.news)
        if n:
            ref = S.attend(self.q[:n], self.k, self.v, self.lens, self.table, self.cu, scale, skip=skip, **self.scales)
            S.check_attend(got[:n], lse[:n], ref, max(self.lens), 11 if self.fp8 else 8)
        assert bool((got[n:] == 77.0).all()) and bool((lse[n:] == 123.0).all())  # rows behind the last request
        return got, lse


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,news", [
    ([1], [1]), ([5], [5]), ([127], [1]), ([128], [1]), ([129], [1]), ([128], [128]), ([129], [129]), ([131], [3]),
    ([300], [7]), ([300], [8]), ([300], [9]), ([300], [15]), ([300], [16]), ([300], [17]), ([520], [136]), ([1000], [33]),
    ([2500], [1]), ([4096], [64]), ([640], [640]),
])
def test_one_request(lens, news, cache):
    Batch(lens, news, cache).poison().check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("seed", range(4))
def test_mixed_batches(seed, cache):
    rng = torch.Generator().manual_seed(seed)

    def draw(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=rng))
    news = [draw(0, 3) if draw(0, 1) else draw(1, 90) for _ in range(draw(2, 40))] + [1]
    lens = [max(m + draw(0, 1200) * draw(0, 1), 0) for m in news]
    Batch(lens, news, cache, seed=seed, width=S.pages(max(lens)) + 3, rows=sum(news) + 5).poison().check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("batch", [1, 7, 33, 150, 400])
def test_single_tokens(batch, cache):
    lens = [1 + (r * 977) % 3001 for r in range(batch)]
    Batch(lens, [1] * batch, cache, seed=batch).poison().check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_every_small_amount_of_work(cache):
    # few blocks for many CTAs: shares at the least size they can have, with items of one and of two tiles
    for blocks in range(1, 13):
        for news in ([9], [1], [16, 1], [3, 12], [2, 2, 11]):
            lens = [max(m, 128 * max(1, blocks // len(news)) - 5 * i) for i, m in enumerate(news)]
            Batch(lens, news, cache, seed=blocks).check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_more_requests_than_threads(cache):
    lens = [1 + (r * 37) % 300 for r in range(1300)]
    news = [min(n, 1 + (r % 7 == 0) + 15 * (r % 50 == 0)) for r, n in enumerate(lens)]
    Batch(lens, news, cache, seed=4).poison().check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [[1, 16, 17, 5], [40, 1, 1, 33], [1, 1, 1, 1]])
def test_values_that_are_not_finite_stay_where_they_are(news, cache):
    # a NaN query reaches its own row; a NaN key or an infinite value the rows of its request and KV head that see it
    b = Batch([700, 500, 300, 200], news, cache, seed=6)
    good = b.call()
    b.q[0, 5, 3] = math.nan
    slot = int(b.table[2, 1]) * 128 + 2  # key 130 of request 2: seen by all its new tokens
    b.k[slot, 1, 7] = torch.tensor(math.nan).to(b.k.dtype)
    got, lse = b.call()
    bad = torch.zeros(b.q.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 5] = True
    at = int(b.cu[2])
    bad[at:at + news[2], 16:32] = True
    assert bool(torch.isnan(got[bad].float()).all()) and bool(torch.isnan(lse[bad]).all())
    assert torch.equal(got[~bad], good[0][~bad]) and torch.equal(lse[~bad], good[1][~bad])


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [[1, 1, 20], [1, 1, 1]])
def test_long_context_is_split_and_joined(news, cache):
    Batch([40000, 3, 17000], news, cache).poison().check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("order", ["up", "down", "one"])
@pytest.mark.parametrize("news", [[40, 1], [1, 1]])
def test_maximum_that_moves(news, order, cache):
    # scores that grow (or fall) from block to block by tens of units, and one key that takes nearly all the weight
    b = Batch([1500, 700], news, cache, seed=5)
    pos = torch.arange(1500, device="cuda")
    size = {"up": pos / 150, "down": 10 - pos / 150, "one": torch.where(pos == 611, 20.0, 0.1)}[order]
    for r in range(2):
        n = b.lens[r]
        slot = b.table[r].long()[pos[:n] // 128] * 128 + pos[:n] % 128
        b.k[slot] = (b.q[0, ::16].float()[None] * size[:n, None, None]).to(b.k.dtype)
    b.check()
    b.check(scale=2.0)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_equal_scores_average_the_values(cache):
    b = Batch([900], [5], cache)
    b.k.zero_()
    b.check()


def test_large_and_small_scales():
    b = Batch([800], [20], seed=3)
    for scale in (1e-6, 0.02, 5.0):
        b.check(scale=scale)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_bad_lengths_and_pages(cache):
    b = Batch([500, 700, 300, 400, 260], [10, 1, 300, 40, 2], cache, seed=2)
    pool = b.k.shape[0] // 128
    ws = msa.Workspace(4096 + msa.workspace_size(msa.make_config(), 4, b.q.shape[0], b.table.shape[1]))
    # request 0: more new tokens than keys; request 1: longer than its table row
    bad = b.seq.clone()
    bad[0], bad[1] = 9, b.table.shape[1] * 128 + 1
    seq, b.seq = b.seq, bad
    got, lse = b.call(workspace=ws)
    assert ws.read_device_error() in ((3, 0), (3, 1))
    assert bool((got[:11] == 0).all()) and bool((lse[:11] == -math.inf).all())
    # the others' rows (where their keys are split follows the whole batch, so not bit for bit those of another batch)
    ref = S.attend(b.q, b.k, b.v, b.lens, b.table, b.cu, SCALE, **b.scales)
    S.check_attend(got[11:], lse[11:], [x[11:] for x in ref], max(b.lens), 11 if b.fp8 else 8)
    b.seq = seq
    # pages outside the pool: their keys are left out
    width = b.table.shape[1]
    b.table[0, 1], b.table[3, 0], b.table[4, 2] = -1, pool, 2 ** 30
    b.check(workspace=ws, skip=((0, 1), (3, 0), (4, 2)))
    assert ws.read_device_error() in ((1, 1), (1, 3 * width), (1, 4 * width + 2))
    # every page bad: rows without a key
    b.table[0, :4] = -5
    got, lse = b.call()
    assert bool((got[:10] == 0).all()) and bool((lse[:10] == -math.inf).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_bad_lengths_and_pages_of_single_tokens(cache):
    b = Batch([500, 700, 300, 400, 260, 0], [1, 1, 1, 1, 1, 0], cache, seed=8).poison()
    width = b.table.shape[1]
    ws = msa.Workspace(4096 + msa.workspace_size(msa.make_config(), 4, b.q.shape[0], width))
    bad = b.seq.clone()
    bad[0], bad[1] = 0, width * 128 + 1
    seq, b.seq = b.seq, bad
    got, lse = b.call(workspace=ws)
    assert ws.read_device_error() in ((3, 0), (3, 1))
    assert bool((got[:2] == 0).all()) and bool((lse[:2] == -math.inf).all())
    ref = S.attend(b.q, b.k, b.v, b.lens, b.table, b.cu, SCALE, **b.scales)
    S.check_attend(got[2:], lse[2:], [x[2:] for x in ref], max(b.lens), 11 if b.fp8 else 8)
    b.seq = seq
    # bad pages, the last (cut inside) among them, and a request without a good one
    b.table[0, 1], b.table[3, 0], b.table[4, 2] = -1, b.k.shape[0] // 128, 2 ** 30
    b.check(workspace=ws, skip=((0, 1), (3, 0), (4, 2)))
    assert ws.read_device_error() in ((1, 1), (1, 3 * width), (1, 4 * width + 2))
    b.table[2, :3] = -5
    got, lse = b.call()
    assert bool((got[2] == 0).all()) and bool((lse[2] == -math.inf).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("news", [[0, 3, 0, 0, 1, 0], [17] + [0] * 10 + [1] * 4 + [0] * 9, [0, 0, 2], [0, 1, 0], [0, 0]])
def test_fewer_tokens_than_requests(news, cache):
    # single tokens alone or beside others, among requests that bring none
    lens = [max(m, 1 + (r * 631) % 1500) for r, m in enumerate(news)]
    Batch(lens, news, cache, seed=len(news), rows=max(sum(news), 1)).poison().check()
    Batch(lens, news, cache, seed=len(news), rows=len(news)).poison().check()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_more_single_tokens_than_threads(cache):
    lens = [1 + (r * 53) % 400 for r in range(1100)]
    Batch(lens, [int(r % 3 > 0) for r in range(1100)], cache, seed=9).poison().check()


def test_unused_table_entries_are_not_read():
    b = Batch([300, 130], [4, 1], width=9)
    want = b.call()
    b.table[0, 3:], b.table[1, 2:] = -7, 2 ** 30
    ws = msa.Workspace(msa.workspace_size(msa.make_config(), 4, b.q.shape[0], 9))
    got = b.call(workspace=ws)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and ws.read_device_error()[0] == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_results_repeat_bitwise(cache):
    b = Batch([9000, 800, 300, 5000], [1, 100, 300, 16], cache)
    a = b.call()
    for _ in range(3):
        c = b.call()
        assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    assert torch.equal(b.call(lse=False)[0], a[0])


def test_two_streams_at_once():
    batches = [Batch([9000 + 50 * i, 800, 300], [1, 100, 30], seed=i) for i in range(2)]
    want = [b.call() for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    for _ in range(20):
        got = []
        for b, s in zip(batches, streams):
            with torch.cuda.stream(s):
                got.append(b.call())
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


def test_captured_graphs_share_nothing():
    # two graphs of different batches, replayed at once; lengths that change between replays
    batches = [Batch([9000, 800, 300], [1, 100, 30], seed=7), Batch([2000, 5000], [1, 1], seed=8)]
    graphs, outs = [], []
    for b in batches:
        b.call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.call())
        graphs.append(g)
    for step in range(3):
        streams = [torch.cuda.Stream() for _ in graphs]
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for b, o in zip(batches, outs):
            want = b.call()
            assert torch.equal(want[0], o[0]) and torch.equal(want[1], o[1])
            b.seq[0] -= 130
            b.lens[0] -= 130


def test_slots_whose_offsets_pass_32_bits():
    # a pool of 2^22 + 256 slots: the last pages begin past 2^32 bytes (and 2^31 elements)
    slots = 2 ** 22 + 256
    k = torch.zeros(slots, 4, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    b = Batch([300, 200], [9, 1])
    last = slots // 128 - 1
    table = torch.tensor([[last, 0, last - 1], [1, last - 2, 0]], dtype=torch.int32, device="cuda")
    for r, n in enumerate(b.lens):
        for p in range(S.pages(n)):
            src, dst = int(b.table[r, p]), int(table[r, p])
            k[dst * 128:dst * 128 + 128] = b.k[src * 128:src * 128 + 128]
            v[dst * 128:dst * 128 + 128] = b.v[src * 128:src * 128 + 128]
    want = b.call()
    b.k, b.v, b.table = k, v, table
    got = b.call()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_agrees_with_the_sparse_decode_when_every_block_is_selected():
    lens = [1, 128, 700, 2048, 1999]
    b = Batch(lens, [1] * 5, seed=11)
    q2k = torch.full((4, 5, 16), -1, dtype=torch.int32, device="cuda")
    for r, n in enumerate(lens):
        q2k[:, r, :S.pages(n)] = torch.arange(S.pages(n), device="cuda")
    got, _ = b.check()
    other = msa.msa_sparse_attend_decode(b.q, b.k, b.v, q2k, b.seq, b.table)
    ref = S.attend(b.q, b.k, b.v, lens, b.table, b.cu, SCALE)
    S.check_attend(other, None, ref, 2048, 8)
