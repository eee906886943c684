"""The int8 K/V cache on the GPU: rows quantised as they are written, read back, and the decode attention over selected blocks,
against 64-bit implementations."""
import math

import pytest
import torch

import _int8kv as ref
import block_sparse_attention_08_gb300 as msa
from _serving import D, G, H, PAGE, ints, offsets, page_table

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(D)


def _bits(x):
    return x.view(torch.int16)


def _insert(k, v, slots, pages, workspace=None):
    """The caches after an insertion, over a pattern that shows what was written."""
    caches = [torch.full((pages * PAGE, G, D), 77, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.full((pages, G, PAGE), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    msa.msa_quantize_insert(k, v, slots, *caches, *scales, workspace=workspace)
    return caches, scales


def _check_insert(x, slots, cache, scales):
    want = torch.full(cache.shape, 77, dtype=torch.int8)
    want_s = torch.full((cache.shape[0], G), 3.0, dtype=torch.float64)
    n, s = ref.quantise(x)
    slots = slots.cpu()
    live = (slots >= 0) & (slots < cache.shape[0])
    want[slots[live]], want_s[slots[live]] = n[live].to(torch.int8), s[live]
    assert torch.equal(cache.cpu(), want)
    got = scales.cpu().double().transpose(1, 2).reshape(-1, G)
    assert torch.equal(got.isnan(), want_s.isnan()) and torch.equal(got.nan_to_num(5.0), want_s.nan_to_num(5.0))


@pytest.mark.parametrize("tokens", [1, 2, 3, 64, 127, 1000, 20000])
def test_insert_equals_the_definition(tokens):
    gen = torch.Generator("cuda").manual_seed(tokens)
    qkv = torch.randn(tokens, 11, D, generator=gen, device="cuda").bfloat16()  # a projection's output: k and v are its heads
    qkv *= torch.exp2(torch.randint(-60, 60, (tokens, 11, 1), generator=gen, device="cuda").float()).bfloat16()
    k, v = qkv[:, 3:7], qkv[:, 7:]
    pages = tokens // PAGE + 3
    slots = torch.randperm(pages * PAGE, generator=gen, device="cuda")[:tokens]
    caches, scales = _insert(k, v, slots, pages)
    for x, c, s in zip((k, v), caches, scales):
        _check_insert(x, slots, c, s)


def test_insert_values_at_the_borders():
    """Zeros, subnormal rows, the largest numbers, ties, halves that saturate, infinities and NaN."""
    rows = torch.zeros(12, G, D)
    rows[1] = 2.0 ** -133 * (torch.arange(D) % 5)                     # subnormals alone
    rows[2, :, 0], rows[2, :, 1:] = 2.0 ** -126, 2.0 ** -133          # the least normal number
    rows[3] = torch.linspace(-1, 1, D) * 3.3e38
    rows[4, :, 0], rows[4, :, 1:] = 64.0, torch.arange(1, D) / 2      # steps of 1: ties to even
    rows[5, :, 0], rows[5, :, 1:] = -64.0, -torch.arange(1, D) / 2
    rows[6] = 127.5                                                   # (a step of 1: 127 at most)
    rows[7], rows[7, :, 5] = 1.0, math.inf
    rows[8], rows[8, 2, 9] = 1.0, math.nan                            # in one head only
    rows[9], rows[9, :, 127] = 2.0 ** -133, -math.inf
    rows[10, :, 3], rows[10, :, 4] = 2.0 ** 100, 2.0 ** -100          # far apart
    rows[11] = -0.0
    x = rows.bfloat16().cuda()
    slots = torch.arange(12, device="cuda") * 3
    caches, scales = _insert(x, -x, slots, 1)
    _check_insert(x, slots, caches[0], scales[0])
    _check_insert(-x, slots, caches[1], scales[1])


def test_insert_skips_rows_and_tells_bad_slots():
    x = torch.randn(300, G, D, device="cuda").bfloat16()
    slots = torch.arange(300, device="cuda") + 100
    slots[::3] = -1
    slots[7] = -(1 << 40)
    ws = msa.Workspace(256)
    caches, scales = _insert(x, x, slots, 4, ws)
    assert ws.read_device_error() == (0, 0)
    _check_insert(x, slots, caches[0], scales[0])
    slots[31] = 4 * PAGE
    caches, scales = _insert(x, x, slots, 4, ws)
    assert ws.read_device_error() == (1, 31)
    _check_insert(x, slots, caches[1], scales[1])
    slots[31] = 1 << 40
    caches, scales = _insert(x, x, slots, 4, ws)
    assert ws.read_device_error() == (1, 31)


def _gather_ref(k, lens_from, table, cu, total, fill):
    out = torch.full((total, G, D), fill, dtype=torch.bfloat16, device="cuda")
    vals = k.bfloat16()
    for r, start in enumerate(lens_from):
        a, b = int(cu[r]), int(cu[r + 1])
        pos = start + torch.arange(b - a, device="cuda")
        page = table[r].long()[(pos // PAGE).clamp(max=table.shape[1] - 1)]
        ok = (page >= 0) & (page < k.shape[0] // PAGE)
        out[a:b] = torch.where(ok[:, None, None], vals[page.clamp(0, k.shape[0] // PAGE - 1) * PAGE + pos % PAGE], 0.0)
    return out


@pytest.mark.parametrize("counts,starts,powers", [
    ([1], [0], True), ([5, 0, 1, 300], [0, 7, 127, 100], True), ([129, 127, 128], [0, 1, 128], False),
    ([0, 0, 2000, 0, 1], None, True), ([3] * 700, [i % 250 for i in range(700)], True)])
def test_gather(counts, starts, powers):
    first = starts or [0] * len(counts)
    table, pages = page_table([s + n for s, n in zip(first, counts)])
    k, ks = ref.cache(pages, 1, powers=powers)
    v, vs = ref.cache(pages, 2, powers=powers)
    cu, total = offsets(counts), sum(counts) + 5
    ko, vo = (torch.full((total, G, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = msa.Workspace(256)
    r = msa.msa_dequantize_gather(k, v, ks, vs, table, cu, total, starts=None if starts is None else ints(starts), k_out=ko,
                                  v_out=vo, workspace=ws)
    assert r[0] is ko and r[1] is vo and ws.read_device_error() == (0, 0)
    # one rounding of an exact product: 15 bits in fp32
    assert torch.equal(ko, _gather_ref(ref.values(k, ks, torch.float32), first, table, cu, total, 9.0))
    assert torch.equal(vo, _gather_ref(ref.values(v, vs, torch.float32), first, table, cu, total, 9.0))


def test_gather_gives_zeros_for_bad_ranges_and_pages():
    counts, first = [10, 200, 5, 5], [0, 0, 0, 0]
    table, pages = page_table([256] * 4, width=2)
    k, ks = ref.cache(pages)
    cu, ws = offsets(counts), msa.Workspace(256)
    for starts, code in (([0, 0, -1, 0], (3, 2)), ([0, 57, 0, 0], (3, 1)), ([0, 0, 0, 2 ** 31 - 1], (3, 3))):
        got, _ = msa.msa_dequantize_gather(k, k, ks, ks, table, cu, 220, starts=ints(starts), workspace=ws)
        assert ws.read_device_error() == code
        want = _gather_ref(ref.values(k, ks, torch.float32), first, table, cu, 220, 0.0)
        a, b = int(cu[code[1]]), int(cu[code[1] + 1])
        want[a:b] = 0
        assert torch.equal(got, want)
    for bad in (-1, pages, 2 ** 31 - 1):
        t = table.clone()
        t[1, 1] = bad
        got, _ = msa.msa_dequantize_gather(k, k, ks, ks, t, cu, 220, workspace=ws)
        assert ws.read_device_error() == (1, 3)
        assert torch.equal(got, _gather_ref(ref.values(k, ks, torch.float32), first, t, cu, 220, 0.0))


def test_rows_that_are_not_finite_read_back_as_nan():
    x = torch.ones(3, G, D, dtype=torch.bfloat16, device="cuda")
    x[1, 2, 5], x[2, 0, 0] = math.inf, math.nan
    caches, scales = _insert(x, x, torch.arange(3, device="cuda"), 1)
    k, _ = msa.msa_dequantize_gather(*caches, *scales, ints([[0]]), ints([0, 3]), 3)
    bad = torch.zeros(3, G, dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[2, 0] = True
    assert bool(k[bad].isnan().all()) and bool((k[~bad] == 1).all())


def _selection(lens, topk, gen):
    q2k = torch.full((G, len(lens), topk), -1, dtype=torch.int32)
    for g in range(G):
        for r, n in enumerate(lens):
            nb = max(1, -(-n // PAGE))
            keep = sorted(torch.randperm(nb - 1, generator=gen)[:topk - 1].tolist() + [nb - 1]) if n else []
            q2k[g, r, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
    return q2k.cuda()


@pytest.mark.parametrize("lens,topk,powers", [
    ([1], 16, True), ([128, 129, 64, 65], 16, True), ([5000], 1, True), ([3000, 17, 2500, 4097], 16, False),
    ([2000 + 37 * i for i in range(40)], 16, True), ([1 + 61 * i for i in range(90)], 7, True)])
def test_sparse_attend(lens, topk, powers):
    gen = torch.Generator().manual_seed(len(lens))
    table, pages = page_table(lens)
    k, ks = ref.cache(pages, 1, powers=powers)
    v, vs = ref.cache(pages, 2, powers=powers)
    # slots behind each request's last key hold scales that are not numbers
    for r, n in enumerate(lens):
        if n % PAGE:
            for s in (ks, vs):
                s[int(table[r, n // PAGE]), :, n % PAGE:] = math.nan if r % 2 else math.inf
    q = torch.randn(len(lens), H, D, generator=gen).bfloat16().cuda()
    q2k = _selection(lens, topk, gen)
    ws = msa.Workspace(256)
    want = ref.sparse(q, ref.values(k, ks), ref.values(v, vs), q2k, lens, table, SCALE)
    for workspace in (None, ws):
        got = msa.msa_sparse_attend_decode_int8kv(q, k, v, ks, vs, q2k, ints(lens), table, workspace=workspace)
        ref.check_sparse(got, want, powers)
    assert ws.read_device_error() == (0, 0)


def test_sparse_attend_bad_blocks_and_pages():
    lens, gen = [1500, 900], torch.Generator().manual_seed(5)
    table, pages = page_table(lens)
    k, ks = ref.cache(pages, 1)
    q = torch.randn(2, H, D, generator=gen).bfloat16().cuda()
    q2k = _selection(lens, 16, gen)
    q2k[:, 1] = -1                                # a row without a block
    table[0, 3] = pages                           # and a page outside the pool
    ws = msa.Workspace(256)
    got = msa.msa_sparse_attend_decode_int8kv(q, k, k, ks, ks, q2k, ints(lens), table, workspace=ws)
    assert ws.read_device_error()[0] == 1
    assert bool((got[1] == 0).all())
    ref.check_sparse(got, ref.sparse(q, ref.values(k, ks), ref.values(k, ks), q2k, lens, table, SCALE))
    q2k[2, 0, 15] = 12                            # a block behind the context
    msa.msa_sparse_attend_decode_int8kv(q, k, k, ks, ks, q2k, ints(lens), table, workspace=ws)
    assert ws.read_device_error()[0] in (1, 2)


def test_sparse_attend_equals_the_bf16_call_on_the_values():
    """Powers of two: the int8 values are bf16 numbers, so both calls attend to the same keys."""
    lens, gen = [4000 + i for i in range(64)], torch.Generator().manual_seed(1)
    table, pages = page_table(lens)
    k, ks = ref.cache(pages, 1)
    v, vs = ref.cache(pages, 2)
    q = torch.randn(64, H, D, generator=gen).bfloat16().cuda()
    q2k = _selection(lens, 16, gen)
    got = msa.msa_sparse_attend_decode_int8kv(q, k, v, ks, vs, q2k, ints(lens), table)
    kb, vb = ref.values(k, ks, torch.float32).bfloat16(), ref.values(v, vs, torch.float32).bfloat16()
    want = msa.msa_sparse_attend_decode(q, kb, vb, q2k, ints(lens), page_table=table)
    # each rounds its weights by 2^-8 in the values' sum and in theirs, and the output by 2^-8
    spread = ref.sparse(q, kb, vb, q2k, lens, table, SCALE)[1]
    assert bool(((got.double() - want.double()).abs() <= 2.0 ** -7 * want.double().abs() + 4 * 2.0 ** -8 * 1.01 * spread).all())


@pytest.mark.parametrize("tokens", [1, 4096, 4097])
def test_new_outputs_are_apart(tokens):
    (k, ks), (v, vs) = ref.cache(2, 1), ref.cache(2, 2)
    table, cu = ints([[i % 2 for i in range(33)]]), ints([0, tokens])
    ko, vo = msa.msa_dequantize_gather(k, v, ks, vs, table, cu, tokens)
    want = vo.clone()
    assert ko.shape == vo.shape == (tokens, G, D) and ko.is_contiguous() and vo.is_contiguous()
    assert ko.data_ptr() % 256 == vo.data_ptr() % 256 == 0
    ko.fill_(3)
    assert torch.equal(vo, want) and bool((ko == 3).all())
    del ko
    torch.cuda.synchronize()
    torch.full((tokens, G, D), 5.0, device="cuda")
    assert torch.equal(vo, want)


def test_new_outputs_are_ordinary_tensors():
    (k, ks), (v, vs) = ref.cache(2, 1), ref.cache(2, 2)
    args = (k, v, ks, vs, ints([[0, 1]]), ints([0, 200]), 200)
    ko, vo = msa.msa_dequantize_gather(*args)
    ko.requires_grad_()
    (ko.float() * vo.float()).sum().backward()
    assert torch.equal(ko.grad, vo) and not vo.requires_grad
    with torch.inference_mode():
        a, b = msa.msa_dequantize_gather(*args)
        assert a.is_inference() and torch.equal(a, ko.detach()) and torch.equal(b, vo)
    rows = vo[3:9].clone()
    vo[3:9].zero_()
    assert bool((vo[3:9] == 0).all()) and bool((rows != 0).any())


@pytest.mark.parametrize("requests", [2, 12, 60])
def test_sparse_attend_names_a_block_behind_the_context(requests):
    """In each launch form, where nothing else is wrong: the block is told, with its place in q2k, and adds no key."""
    lens, gen = [1500 + r for r in range(requests)], torch.Generator().manual_seed(6)
    table, pages = page_table(lens, width=20)      # (entries behind a request's pages name page 0: what is there must not count)
    k, ks = ref.cache(pages, 1)
    v, vs = ref.cache(pages, 2)
    q = torch.randn(requests, H, D, generator=gen).bfloat16().cuda()
    ws = msa.Workspace(256)
    for r, g, j, block in ((requests - 1, 2, 15, 12 + (requests > 36)), (0, 0, 5, 19), (1, 3, 0, 2 ** 31 - 1)):
        q2k = _selection(lens, 16, gen)
        q2k[g, r, j] = block
        got = msa.msa_sparse_attend_decode_int8kv(q, k, v, ks, vs, q2k, ints(lens), table, workspace=ws)
        # detail: the entry's number, request by request
        assert ws.read_device_error() == (2, (r * G + g) * 16 + j)
        ref.check_sparse(got, ref.sparse(q, ref.values(k, ks), ref.values(v, vs), q2k, lens, table, SCALE))
