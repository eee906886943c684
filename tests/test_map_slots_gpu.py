"""Page-table rows and slot maps on the GPU against a request-by-request implementation: whole numbers, equal."""
import random

import pytest
import torch

import _serving as S
import block_sparse_attention_08_gb300 as msa

pytestmark = pytest.mark.gpu


def _run(lens, news, table, free, num_free, num_slots, capacity, ws=None):
    t = torch.tensor(table, dtype=torch.int32, device="cuda")
    f = torch.tensor(free, dtype=torch.int32, device="cuda")
    cu, slots, positions, left = msa.msa_map_slots(S.ints(lens), S.ints(news), t, f, S.ints([num_free]),
                                                   num_slots=num_slots, capacity=capacity, workspace=ws)
    return cu.tolist(), slots.tolist(), positions.tolist(), t.tolist(), int(left)


def _case(seed, batch, longest, fresh, spare_pages=3):
    rng = random.Random(seed)
    news = [min(rng.choice([0, 1, 1, 2, rng.randint(0, fresh)]), longest) for _ in range(batch)]
    lens = [rng.randint(max(m, 0), longest) for m in news]
    have = [S.pages(n - m) for n, m in zip(lens, news)]
    opened = sum(S.pages(n) for n in lens) - sum(have)
    ids = list(range(sum(have) + opened + spare_pages))
    rng.shuffle(ids)
    width = max(S.pages(n) for n in lens) + rng.randint(0, 2)
    table = [[ids.pop() for _ in range(h)] + [7] * (max(width, 1) - h) for h in have]
    return lens, news, table, ids, len(ids), (sum(have) + len(ids)) * S.PAGE


@pytest.mark.parametrize("batch,longest,fresh", [(1, 1, 1), (1, 128, 128), (3, 129, 129), (64, 65536, 1), (17, 5000, 700),
                                                 (511, 900, 30), (512, 300, 9), (513, 300, 9), (2000, 1000, 40),
                                                 (1, 131072, 131072), (2, 20000, 20000)])
def test_against_the_plain_form(batch, longest, fresh):
    for seed in range(3):
        lens, news, table, free, num_free, slots = _case(seed, batch, longest, fresh)
        for spare in (0, 5, 3000):
            capacity = max(1, sum(news) + spare)
            ws = msa.Workspace(256)
            *want, errors = S.map_slots(lens, news, table, free, num_free, slots, capacity)
            assert not errors
            assert _run(lens, news, table, free, num_free, slots, capacity, ws) == tuple(want)
            assert ws.read_device_error()[0] == 0


def test_whole_pages_and_their_borders():
    # old and new lengths on, before and after a page's border
    lens = [128, 128, 129, 256, 257, 127, 1, 0, 384, 130]
    news = [1, 128, 1, 128, 129, 0, 1, 0, 256, 3]
    have = [S.pages(n - m) for n, m in zip(lens, news)]
    table = [list(range(10 * r, 10 * r + h)) + [0] * (3 - h) for r, h in enumerate(have)]
    free = list(range(200, 220))
    *want, errors = S.map_slots(lens, news, table, free, 15, 300 * 128, 700)
    assert not errors and _run(lens, news, table, free, 15, 300 * 128, 700) == tuple(want)


@pytest.mark.parametrize("seed", range(6))
def test_what_does_not_fit_maps_nothing(seed):
    rng = random.Random(seed)
    lens, news, table, free, num_free, slots = _case(seed, 700, 2000, 300)
    if seed % 2:
        num_free = rng.randint(0, num_free)  # pages run out
        capacity = sum(news)
    else:
        capacity = max(1, rng.randint(0, sum(news)))
    ws = msa.Workspace(256)
    *want, errors = S.map_slots(lens, news, table, free, num_free, slots, capacity)
    assert _run(lens, news, table, free, num_free, slots, capacity, ws) == tuple(want)
    code = ws.read_device_error()
    assert (code in errors) if errors else code[0] == 0


def test_bad_lengths_and_pages_are_reported():
    lens, news, table, free, num_free, slots = _case(9, 40, 3000, 200)
    lens[3], news[3] = 10, 11                      # more new tokens than tokens
    news[7] = -1
    lens[11] = len(table[11]) * S.PAGE + 1         # longer than its table row
    for num in (num_free, len(free) + 1, -3):      # the last two count as an empty stack
        ws = msa.Workspace(256)
        *want, errors = S.map_slots(lens, news, table, free, num, slots, sum(max(n, 0) for n in news))
        got = _run(lens, news, table, free, num, slots, sum(max(n, 0) for n in news), ws)
        if 0 <= num <= len(free):
            assert got == tuple(want)
        else:
            assert got[:4] == tuple(want[:4]) and got[4] == 0
        assert ws.read_device_error() in errors
    # a page id outside the pool: from the table, and from the stack
    lens, news, table, free = [200, 300], [72, 300], [[900, 0, 0], [0, 0, 0]], [4, 5, 6, -2, 7]
    ws = msa.Workspace(256)
    *want, errors = S.map_slots(lens, news, table, free, 5, 20 * S.PAGE, 400)
    assert _run(lens, news, table, free, 5, 20 * S.PAGE, 400, ws) == tuple(want)
    assert ws.read_device_error() in errors


def test_repeated_and_captured_calls_agree():
    lens, news, table, free, num_free, slots = _case(4, 100, 4000, 500)
    args = [S.ints(lens), S.ints(news), torch.tensor(table, dtype=torch.int32, device="cuda"),
            torch.tensor(free, dtype=torch.int32, device="cuda"), S.ints([num_free])]
    kw = dict(num_slots=slots, capacity=sum(news) + 10)
    first = [x.clone() for x in msa.msa_map_slots(*args, **kw)] + [args[2].clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        msa.msa_map_slots(*args, **kw)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = msa.msa_map_slots(*args, **kw)
    for x in out:
        x.fill_(99)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, list(out) + [args[2]]))


def test_more_rows_than_threads_at_once():
    # beyond 4 * 152 CTAs of 512 threads a CTA takes several passes over its rows; requests begin inside them
    lens = [400_000, 5, 300_001, 0, 129, 131_072]
    news = [400_000, 3, 299_999, 0, 1, 131_072]
    have = [S.pages(n - m) for n, m in zip(lens, news)]
    width = max(S.pages(n) for n in lens)
    opened = sum(S.pages(n) for n in lens) - sum(have)
    ids = list(range(sum(have) + opened + 2))
    random.Random(1).shuffle(ids)
    table = [[ids.pop() for _ in range(h)] + [0] * (width - h) for h in have]
    slots = (sum(have) + len(ids)) * S.PAGE
    for capacity in (sum(news), sum(news) + 70_001):
        *want, errors = S.map_slots(lens, news, table, ids, len(ids), slots, capacity)
        assert not errors and _run(lens, news, table, ids, len(ids), slots, capacity) == tuple(want)


def test_outputs_given_and_new_agree():
    # new outputs are parts of one allocation: whole tensors to their user all the same
    lens, news, table, free, num_free, num_slots = _case(5, 9, 700, 90)
    t = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (table, free)]
    args = S.ints(lens), S.ints(news), t[0], t[1], S.ints([num_free])
    sizes = {"num_slots": num_slots, "capacity": sum(news) + 3}
    new = msa.msa_map_slots(*args, **sizes)
    given = [torch.full_like(x, 5) for x in new]
    out = msa.msa_map_slots(*args, **sizes, **dict(zip(("cu_seqlens_q", "slots", "positions", "num_free_out"), given)))
    for a, b, c in zip(new, out, given):
        assert torch.equal(a, b) and torch.equal(a, c) and b.data_ptr() == c.data_ptr()
        assert a.is_contiguous() and a.clone().tolist() == a.tolist()
    # writing one leaves the others
    keep = [x.clone() for x in new]
    for i, x in enumerate(new):
        x.fill_(-9)
        assert all(torch.equal(a, b) for a, b in zip(new[i + 1:], keep[i + 1:]))
