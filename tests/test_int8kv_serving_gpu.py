"""The int8 cache's calls and the attention over shared prefixes together, as a program calls them: in a serving loop, captured,
from several threads, on long caches."""
import math
import threading

import pytest
import torch

import _int8kv as i8
import _serving as S
import block_sparse_attention_08_gb300 as msa

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(128.0)


def _cache(pages, value=77):
    """A cache that shows what has not been written: its rows are not finite."""
    return ([torch.full((pages * 128, 4, 128), value, dtype=torch.int8, device="cuda") for _ in range(2)] +
            [torch.full((pages, 4, 128), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)])


def _quantised(x):
    n, s = i8.quantise(x)
    return (n * s[..., None]).cuda()


def test_a_prompt_answered_nine_times():
    """One request's prompt arrives in two chunks, eight others take over its whole pages and bring the rest of it, and all
    answer with one to three tokens a step; then the sparse decode over the same cache, and the contexts read back."""
    gen = torch.Generator("cuda").manual_seed(1)
    B, width, pool, common = 9, 5, 40, 256
    inv_freq = torch.tensor([1e4 ** (-j / 32) for j in range(32)], device="cuda")
    caches = _cache(pool)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pool, generator=gen, device="cuda", dtype=torch.int32)
    left = S.ints([pool])
    ws = msa.Workspace(msa.workspace_size(msa.make_config(), msa.binding.MODE_SHARED, 512, width))
    lens = [0] * B
    keys, vals = [[torch.empty(0, 4, 128, device="cuda", dtype=torch.float64)] * 2 for _ in range(2)]
    keys, vals = [keys[0] for _ in range(B)], [vals[0] for _ in range(B)]  # what each request's context stands for
    steps = [[200] + [0] * 8, [97] + [0] * 8, [0] + [41] * 8, [1] * 9, [1, 2, 1, 3, 1, 1, 2, 1, 1], [1] * 9, [1, 0, 1, 1, 1, 1, 0, 1, 1]]
    for step, news in enumerate(steps):
        if step == 2:  # the prompt's two whole pages
            lens[1:], keys[1:], vals[1:] = [common] * 8, [keys[0][:common]] * 8, [vals[0][:common]] * 8
            table[1:, :2] = table[:1, :2]
        lens = [n + m for n, m in zip(lens, news)]
        total, cap = sum(news), sum(news) + 3
        cu, slots, pos, left = msa.msa_map_slots(S.ints(lens), S.ints(news), table, free, left, num_slots=pool * 128, capacity=cap,
                                                 workspace=ws)
        qkv = torch.randn(cap, 72, 128, generator=gen, device="cuda").bfloat16()
        q, k = msa.msa_rotary(qkv[:, :64], qkv[:, 64:68], pos, inv_freq)
        msa.msa_quantize_insert(k, qkv[:, 68:], slots, *caches, workspace=ws)
        lse = torch.empty(cap, 64, device="cuda")
        args = (q, *caches, S.ints(lens), table, cu)
        if step < 2:
            out = msa.msa_attend_chunk_int8kv(*args, lse=lse, workspace=ws)
        else:
            out = msa.msa_attend_shared_int8kv(*args, S.ints([0, B]), S.ints([common]), lse=lse, workspace=ws)
        assert ws.read_device_error()[0] == 0 and cu.tolist() == S.offsets(news).tolist()
        new_k, new_v = _quantised(k[:total]), _quantised(qkv[:total, 68:])
        for r, (a, b) in enumerate(zip(cu.tolist(), cu.tolist()[1:])):
            keys[r], vals[r] = torch.cat([keys[r], new_k[a:b]]), torch.cat([vals[r], new_v[a:b]])
        # the contexts as the test keeps them, not as the cache has them
        rows = S.offsets(lens).tolist()
        at = torch.zeros(B, width, dtype=torch.int32, device="cuda")
        kept = [torch.zeros(B * width * 128, 4, 128, dtype=torch.float64, device="cuda") for _ in range(2)]
        for r in range(B):
            at[r] = torch.arange(width, device="cuda") + r * width
            for x, y in zip(kept, (keys[r], vals[r])):
                x[r * width * 128:r * width * 128 + lens[r]] = y
        ref = S.attend(q[:total], *kept, lens, at, cu, SCALE)
        S.check_attend(out[:total], lse[:total], ref, max(lens), 8)
        got = msa.msa_dequantize_gather(*caches, table, S.offsets(lens), rows[-1], workspace=ws)
        assert ws.read_device_error()[0] == 0
        assert torch.equal(got[0].double(), torch.cat(keys)) and torch.equal(got[1].double(), torch.cat(vals))
    index_cache = torch.zeros(pool * 128, 1, 128, dtype=torch.bfloat16, device="cuda")
    iq, qd = (torch.randn(B, h, 128, generator=gen, device="cuda").bfloat16() for h in (4, 64))
    q2k = msa.msa_select_blocks_decode(iq, index_cache, S.ints(lens), page_table=table.clamp(min=0))
    out = msa.msa_sparse_attend_decode_int8kv(qd, *caches, q2k, S.ints(lens), table, workspace=ws)
    assert ws.read_device_error()[0] == 0
    i8.check_sparse(out, i8.sparse(qd, *kept, q2k, lens, at, SCALE))


def _step(x, caches, inv, seq, new, table, free, left, pool, cap, off, shared, ws=None):
    cu, slots, pos, now = msa.msa_map_slots(seq, new, table, free, left, num_slots=pool * 128, capacity=cap, workspace=ws)
    q, k = msa.msa_rotary(x[:, :64], x[:, 64:68], pos, inv)
    msa.msa_quantize_insert(k, x[:, 68:], slots, *caches, workspace=ws)
    out = msa.msa_attend_shared_int8kv(q, *caches, seq, table, cu, off, shared, workspace=ws)
    left.copy_(now)
    return q, out, cu


def test_a_captured_step_refilled_between_replays():
    gen = torch.Generator("cuda").manual_seed(5)
    B, width, common = 10, 4, 128
    pool, cap = B * width, 40
    seq, new, left = S.ints([common + 40] * B), S.ints([common + 40] + [40] * (B - 1)), S.ints([pool])
    table, free = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), torch.randperm(pool, generator=gen, device="cuda").int()
    off, shared = S.ints([0, B]), S.ints([common])
    caches, inv = _cache(pool), torch.rand(64, generator=gen, device="cuda")
    ws = msa.Workspace(msa.workspace_size(msa.make_config(), msa.binding.MODE_SHARED, 600, width))
    # the prefix, then the rest of each prompt
    first = S.ints([common] + [0] * (B - 1))
    _step(torch.randn(common, 72, 128, generator=gen, device="cuda").bfloat16(), caches, inv, first, first, table, free, left, pool, common,
          off, S.ints([0]), ws)
    table[1:, 0] = table[0, 0]
    new.fill_(40)
    _step(torch.randn(40 * B, 72, 128, generator=gen, device="cuda").bfloat16(), caches, inv, seq, new, table, free, left, pool, 40 * B, off,
          shared, ws)
    assert ws.read_device_error()[0] == 0
    qkv = torch.empty(cap, 72, 128, dtype=torch.bfloat16, device="cuda")
    new.fill_(1), qkv.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, out, cu = _step(qkv, caches, inv, seq, new, table, free, left, pool, cap, off, shared, ws)
    lens, live = [common + 40] * B, common
    for news, live in (([1] * B, common), ([1] * B, 0), ([1, 4] * 5, common), ([3, 0, 9, 1, 1] * 2, common), ([1] * B, common)):
        lens = [n + m for n, m in zip(lens, news)]
        seq.copy_(S.ints(lens)), new.copy_(S.ints(news)), shared.fill_(live)
        qkv.copy_(torch.randn(cap, 72, 128, generator=gen, device="cuda"))
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert ws.read_device_error()[0] == 0 and cu.tolist() == S.offsets(news).tolist()
        t = sum(news)
        ref = S.attend(q[:t], i8.values(caches[0], caches[2]), i8.values(caches[1], caches[3]), lens, table, cu, SCALE)
        S.check_attend(out[:t], None, ref, max(lens), 8)
        assert bool((out[t:] == 7).all())


def test_calls_from_several_threads_at_once():
    def work(seed):
        gen = torch.Generator("cuda").manual_seed(seed)
        lens, news = [700 + 300 * seed, 640, 3001] + [700 + i for i in range(9)], [1 + 5 * seed, 1, 17] + [1] * 9
        table, pool = S.page_table(lens, seed=seed)
        table[4:, :5] = table[3, :5]
        cu, t = S.offsets(news), sum(news)
        x = torch.randn(t, 72, 128, generator=gen, device="cuda").bfloat16()
        caches = [torch.randint(-127, 128, (pool * 128, 4, 128), generator=gen, device="cuda", dtype=torch.int8) for _ in range(2)]
        caches += [torch.rand(pool, 4, 128, generator=gen, device="cuda").bfloat16() for _ in range(2)]
        slots = torch.randperm(pool * 128, generator=gen, device="cuda")[:t]
        q2k = torch.arange(6, device="cuda", dtype=torch.int32).expand(4, len(lens), 6).contiguous()
        rows, n = S.offsets(lens), sum(lens)
        out = []
        for _ in range(12):
            msa.msa_quantize_insert(x[:, 64:68], x[:, 68:], slots, *caches)
            q = x[:, :64].contiguous()
            out += [*[c.clone() for c in caches], *msa.msa_dequantize_gather(*caches, table, rows, n),
                    msa.msa_attend_chunk_int8kv(q, *caches, S.ints(lens), table, cu),
                    msa.msa_attend_shared_int8kv(q, *caches, S.ints(lens), table, cu, S.ints([3, len(lens)]), S.ints([640])),
                    msa.msa_sparse_attend_decode_int8kv(q[:len(lens)].contiguous(), *caches, q2k, S.ints(lens), table)]
        torch.cuda.current_stream().synchronize()
        return out

    want, got = [work(i) for i in range(4)], [None] * 4

    def on_thread(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = work(i)
        except BaseException as e:  # told on the test's thread
            got[i] = e
    torch.cuda.synchronize()
    threads = [threading.Thread(target=on_thread, args=(i,)) for i in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    for w, g in zip(want, got):
        assert not isinstance(g, BaseException), g
        assert len(w) == len(g) and all(torch.equal(a, b) for a, b in zip(w, g))


def test_one_slot_given_twice():
    """The slot gets either row's values, or some of each: no other row changes."""
    x = torch.randn(64, 8, 128, generator=torch.Generator("cuda").manual_seed(2), device="cuda").bfloat16()
    slots = torch.arange(64, device="cuda")
    slots[40] = 7
    caches, ws = _cache(2), msa.Workspace(256)
    msa.msa_quantize_insert(x[:, :4], x[:, 4:], slots, *caches, workspace=ws)
    assert ws.read_device_error()[0] == 0
    n, s = i8.quantise(x)
    for c, sc, part in ((caches[0], caches[2], slice(0, 4)), (caches[1], caches[3], slice(4, 8))):
        rows = [i for i in range(64) if i not in (7, 40)]
        assert torch.equal(c.cpu()[rows].long(), n[rows, part])
        got = sc.transpose(1, 2).reshape(-1, 4).cpu().double()
        assert torch.equal(got[rows], s[rows, part]) and bool(got[[40] + list(range(64, 256))].isnan().all())
        a, b = n[7, part], n[40, part]
        here = c.cpu()[7].long()
        assert bool(((here == a) | (here == b)).all()) and bool(((got[7] == s[7, part]) | (got[7] == s[40, part])).all())


def _at16(shape):
    """An output that begins on 16 bytes, not on 32."""
    return torch.empty(math.prod(shape) + 8, dtype=torch.bfloat16, device="cuda")[8:].view(shape)


def test_outputs_that_begin_on_16_bytes():
    lens, news = [900, 700] + [650 + i for i in range(9)], [1, 30] + [1] * 9
    table, pool = S.page_table(lens)
    table[3:, :5] = table[2, :5]
    (k, ks), (v, vs) = i8.cache(pool, 1), i8.cache(pool, 2)
    caches = (k, v, ks, vs)
    q = torch.randn(sum(news), 64, 128, generator=torch.Generator("cuda").manual_seed(3), device="cuda").bfloat16()
    args = (q, *caches, S.ints(lens), table, S.offsets(news))
    group = (S.ints([2, 11]), S.ints([640]))
    q2k = torch.arange(6, device="cuda", dtype=torch.int32).expand(4, 11, 6).contiguous()
    for call in (lambda out: msa.msa_attend_chunk_int8kv(*args, out=out), lambda out: msa.msa_attend_shared_int8kv(*args, *group, out=out)):
        assert torch.equal(call(None), call(_at16(q.shape)))
    d = q[:11].contiguous()
    assert torch.equal(msa.msa_sparse_attend_decode_int8kv(d, *caches, q2k, S.ints(lens), table),
                       msa.msa_sparse_attend_decode_int8kv(d, *caches, q2k, S.ints(lens), table, out=_at16(d.shape)))
    rows = S.offsets(lens)
    want = msa.msa_dequantize_gather(*caches, table, rows, sum(lens))
    ko, vo = _at16(want[0].shape), _at16(want[1].shape)
    msa.msa_dequantize_gather(*caches, table, rows, sum(lens), k_out=ko, v_out=vo)
    assert torch.equal(ko, want[0]) and torch.equal(vo, want[1])


def test_offsets_beyond_32_bits():
    """8.4 million slots (4.3 GB a cache), 4.2 million rows read back (4.3 GB an output) and written again."""
    gen = torch.Generator("cuda").manual_seed(4)
    pages, rows = 1 << 16, (1 << 22) + 333
    width = S.pages(rows)
    k, v = (torch.randint(-127, 128, (pages * 128, 4, 128), generator=gen, device="cuda", dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(-7, -4, (pages, 4, 128), generator=gen, device="cuda").float()).bfloat16() for _ in range(2))
    table = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)[None, :width].contiguous()
    table[0, -1] = pages - 1  # the last rows lie behind every 32-bit offset
    ws = msa.Workspace(256)
    ko, vo = msa.msa_dequantize_gather(k, v, ks, vs, table, S.ints([0, rows]), rows, workspace=ws)
    assert ws.read_device_error()[0] == 0
    look = torch.cat([torch.arange(rows - 400, rows, device="cuda"), torch.randint(0, rows, (1000,), generator=gen, device="cuda")])
    slot = table[0].long()[look // 128] * 128 + look % 128

    def value(c, s):
        return c[slot].double() * s.transpose(1, 2)[slot // 128, slot % 128].double()[..., None]
    assert torch.equal(ko[look].double(), value(k, ks)) and torch.equal(vo[look].double(), value(v, vs))
    # the attention over the last pages, by one token and by some, and the sparse one
    near = table[:, -5:].contiguous()
    lens = [4 * 128 + 77]
    for n in (1, 20):
        q = torch.randn(n, 64, 128, generator=gen, device="cuda").bfloat16()
        out = msa.msa_attend_chunk_int8kv(q, k, v, ks, vs, S.ints(lens), near, S.offsets([n]))
        pos = torch.arange(5 * 128, device="cuda")
        at = near[0].long()[pos // 128] * 128 + pos % 128
        small = [c[at].double() * s.transpose(1, 2)[at // 128, at % 128].double()[..., None] for c, s in ((k, ks), (v, vs))]
        flat = S.ints([[0, 1, 2, 3, 4]])
        S.check_attend(out, None, S.attend(q, *small, lens, flat, S.offsets([n]), SCALE), lens[0], 8)
    q, q2k = q[:1].contiguous(), S.ints([0, 3, 4]).expand(4, 1, 3).contiguous()
    out = msa.msa_sparse_attend_decode_int8kv(q, k, v, ks, vs, q2k, S.ints(lens), near, workspace=ws)
    assert ws.read_device_error()[0] == 0
    i8.check_sparse(out, i8.sparse(q, *small, q2k, lens, flat, SCALE))
    # written again elsewhere, from the packed rows
    to = torch.randperm(pages * 128, generator=gen, device="cuda")[:rows]
    to[-1] = pages * 128 - 1 if not bool((to == pages * 128 - 1).any()) else to[-1]
    msa.msa_quantize_insert(ko, vo, to, k, v, ks, vs, workspace=ws)
    assert ws.read_device_error()[0] == 0
    slot = to[look]
    assert torch.equal(ko[look].double(), value(k, ks)) and torch.equal(vo[look].double(), value(v, vs))


@pytest.mark.parametrize("requests", [1, 7, 20, 45, 150])
def test_a_captured_sparse_step_with_lengths_that_change(requests):
    """Split over clusters, and with a CTA for each of few or many segments; requests of no keys at all among them."""
    gen = torch.Generator().manual_seed(requests)
    lens = [1500 + 11 * i % 700 for i in range(requests)]
    table, pool = S.page_table(lens, seed=requests)
    (k, ks), (v, vs) = i8.cache(pool, 1), i8.cache(pool, 2)
    q = torch.randn(requests, 64, 128, generator=gen).bfloat16().cuda()
    q2k = torch.randint(0, 11, (4, requests, 1), generator=gen, dtype=torch.int32).cuda() + torch.arange(6, dtype=torch.int32, device="cuda")
    q2k = torch.where(q2k < 11, q2k, -1).contiguous()
    seq, ws, out = S.ints(lens), msa.Workspace(256), torch.empty_like(q)
    values = i8.values(k, ks), i8.values(v, vs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.msa_sparse_attend_decode_int8kv(q, k, v, ks, vs, q2k, seq, table, out=out, workspace=ws)
    for turn in range(3):
        now = [n if turn == 0 else 1408 + n % 90 if (r + turn) % 3 else 0 for r, n in enumerate(lens)]
        seq.copy_(S.ints(now))
        out.fill_(9)
        # (blocks behind a request's last are an error: none is asked for but by those without keys)
        live = torch.where((torch.tensor(now) > 0)[None, :, None].cuda(), q2k, -1)
        kept = q2k.clone()
        q2k.copy_(live)
        graph.replay()
        torch.cuda.synchronize()
        assert ws.read_device_error()[0] == 0
        i8.check_sparse(out, i8.sparse(q, *values, q2k, now, table, SCALE))
        assert all(bool((out[r] == 0).all()) for r, n in enumerate(now) if n == 0)
        q2k.copy_(kept)
