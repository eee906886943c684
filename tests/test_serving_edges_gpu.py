"""Calls of the chunk-serving functions at the borders of what they accept: addresses, threads, frequencies, lengths,
buffers that change behind autograd."""
import ctypes
import math
import subprocess
import threading
from fractions import Fraction

import pytest
import torch

import _serving as S
import block_sparse_attention_08_gb300 as msa

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(128.0)


def _batch(lens, news, fp8, seed=0):
    """(the call, its tensors): q, k_cache, v_cache, seq_lens, page_table, cu_seqlens_q."""
    gen = torch.Generator("cuda").manual_seed(seed)
    table, pool = S.page_table(lens, seed=seed)
    q = torch.randn(sum(news), 64, 128, generator=gen, device="cuda").bfloat16()
    k, v = (torch.randn(pool * 128, 4, 128, generator=gen, device="cuda").to(torch.float8_e4m3fn if fp8 else torch.bfloat16)
            for _ in range(2))
    return (msa.msa_attend_chunk_fp8kv if fp8 else msa.msa_attend_chunk), [q, k, v, S.ints(lens), table, S.offsets(news)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,news", [([300], [40]), ([9000, 200], [1, 9]), ([500, 40, 7], [1, 1, 1])])
def test_outputs_that_begin_on_16_bytes(lens, news, fp8):
    # whole items of one and of two tiles, cut items, single tokens: the same bits wherever out begins
    call, args = _batch(lens, news, fp8)
    want = call(*args)
    for at in (0, 8, 16, 24):
        room = torch.full((want.numel() + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
        out = room[at:at + want.numel()].view(want.shape)
        assert out.data_ptr() % 32 == 2 * at % 32
        assert call(*args, out=out) is out
        assert torch.equal(out, want)
        assert bool((room[:at] == 5).all()) and bool((room[at + want.numel():] == 5).all())


HAMMER = r"""
#include <pthread.h>
typedef int (*rotary_t)(const void*, const void*, long long, int, const void*, long long, int, const void*, const void*,
                        long long, int, void*, void*, void*);
typedef struct { rotary_t f; const void *rot, *q, *k, *positions, *inv_freq; void *qo, *ko, *stream;
                 int q_heads, k_heads, tokens, times, refused; } call;
static void* work(void* p) {
  call* c = p;
  for (int i = 0; i < c->times; ++i)
    c->refused += c->f(c->rot, c->q, 128 * c->q_heads, c->q_heads, c->k, 128 * c->k_heads, c->k_heads, c->positions,
                       c->inv_freq, c->tokens, 0, c->qo, c->ko, c->stream) != 0;
  return 0;
}
void hammer(call* c, int n) {
  pthread_t t[8];
  for (int i = 0; i < n; ++i) pthread_create(&t[i], 0, work, &c[i]);
  for (int i = 0; i < n; ++i) pthread_join(t[i], 0);
}
"""


class _Call(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("f", "rot", "q", "k", "positions", "inv_freq", "qo", "ko", "stream")] + \
               [(n, ctypes.c_int) for n in ("q_heads", "k_heads", "tokens", "times", "refused")]


def test_rotary_of_different_head_counts_from_several_threads(tmp_path):
    # shared memory of 2, 72 and 128 KB in turn; without the interpreter between the calls
    (tmp_path / "hammer.c").write_text(HAMMER)
    subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-pthread", str(tmp_path / "hammer.c"), "-o", str(tmp_path / "h.so")],
                   check=True)
    hammer = ctypes.CDLL(str(tmp_path / "h.so")).hammer
    lib = msa.load()
    rot = msa.binding.msa_rotary_config(128, 0, 1)
    gen = torch.Generator("cuda").manual_seed(0)
    pos = torch.randint(1000, (5,), generator=gen, device="cuda", dtype=torch.int32)
    inv = torch.rand(64, generator=gen, device="cuda")
    heads = ((1, 1), (64, 64), (64, 4))
    calls, data, streams = (_Call * 3)(), [], [torch.cuda.Stream() for _ in heads]
    for c, s, (qh, kh) in zip(calls, streams, heads):
        x = [torch.randn(5, h, 128, generator=gen, device="cuda").bfloat16() for h in (qh, kh)]
        y = [torch.empty_like(a) for a in x]
        data.append((x, y))
        c.f = ctypes.cast(lib.msa_rotary, ctypes.c_void_p).value
        c.rot = ctypes.addressof(rot)
        c.q, c.k, c.qo, c.ko = (a.data_ptr() for a in x + y)
        c.positions, c.inv_freq, c.stream = pos.data_ptr(), inv.data_ptr(), s.cuda_stream
        c.q_heads, c.k_heads, c.tokens, c.times = qh, kh, 5, 500
    torch.cuda.synchronize()
    for _ in range(20):
        hammer(calls, 3)
        torch.cuda.synchronize()
    assert [c.refused for c in calls] == [0, 0, 0]
    for x, y in data:
        assert all(torch.equal(a, b) for a, b in zip(msa.msa_rotary(*x, pos, inv), y))


def test_angles_of_any_position_and_frequency():
    # (cos, sin) against whole-number arithmetic.  Tolerance: half a bf16 step of the value, 2^-8, and the angle: 2^-24 of a
    # turn is 2^-21.3 in the value, the functions' and the rotation's own errors below 2^-22: 2^-20.5 in all.
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")
    inv = torch.tensor([2.0 ** e for e in (-30, -10, -3, -1, 0)] + [1.5, 3.7, 100.0, 9876.54321, 1e6, 1.23e9, 2.0 ** 32],
                       device="cuda")
    inv = torch.cat([inv, inv[:4] * 0.777])  # 16 pairs
    gen = torch.Generator().manual_seed(0)
    positions = [0, 1, -1, 2 ** 24 - 1, 2 ** 24, 2 ** 24 + 1, -2 ** 24, 2 ** 31 - 1, -2 ** 31]
    positions += [int(torch.randint(2 ** (e - 1), 2 ** e, (1,), generator=gen)) for e in range(2, 32) for _ in range(6)]
    x = torch.zeros(len(positions), 1, 128, dtype=torch.bfloat16, device="cuda")
    x[..., :16] = 1
    y = msa.msa_rotary(x, None, S.ints(positions), inv)[0][:, 0].double().cpu()
    for t, p in enumerate(positions):
        for j, f in enumerate(inv.tolist()):
            turns = p * Fraction(f) / two_pi
            angle = float((turns - round(turns)) * two_pi)
            for got, want in ((y[t, j], math.cos(angle)), (y[t, j + 16], math.sin(angle))):
                assert abs(float(got) - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -20.5, (p, f)


def test_positions_refilled_before_the_backward_are_noticed():
    # a buffer of positions that the next slot map writes: the rotation back would turn by the wrong angles
    table, free, num = S.ints([[0, 1]]), S.ints([0, 1]), S.ints([2])
    new = msa.msa_map_slots(S.ints([9]), S.ints([9]), table, free, num, num_slots=256, capacity=9)
    again = dict(zip(("cu_seqlens_q", "slots", "positions", "num_free_out"), new))
    q, k = (torch.ones(9, h, 128, device="cuda").bfloat16().requires_grad_() for h in (64, 4))
    inv = torch.full((64,), 0.01, device="cuda")
    out = msa.rotary(q, k, new[2], inv)
    grads = [torch.ones_like(x) for x in out]
    torch.autograd.grad(out, (q, k), grads)
    out = msa.rotary(q, k, new[2], inv)
    msa.msa_map_slots(S.ints([200]), S.ints([9]), table, free, num, num_slots=256, capacity=9, **again)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(out, (q, k), grads)
    # a refused call changes nothing
    out = msa.rotary(q, k, new[2], inv)
    with pytest.raises(msa.MsaError):
        msa.msa_map_slots(S.ints([200]), S.ints([9]), table, free, num, num_slots=100, capacity=9, **again)
    torch.autograd.grad(out, (q, k), grads)


@pytest.mark.parametrize("fp8", [False, True])
def test_tensors_that_a_call_writes_are_marked_as_changed(fp8):
    q, k = torch.ones(3, 64, 128, device="cuda").bfloat16(), torch.ones(3, 4, 128, device="cuda").bfloat16()
    inv, pos, slots = torch.full((64,), 0.01, device="cuda"), S.ints([0, 1, 2]), torch.arange(3, device="cuda")
    caches = [torch.zeros(128, 4, 128, device="cuda").to(torch.float8_e4m3fn if fp8 else torch.bfloat16) for _ in range(2)]
    table, cu, lens = S.ints([[0]]), S.ints([0, 3]), S.ints([3])
    lse = torch.empty(3, 64, device="cuda")
    qo, ko, out = q.clone(), k.clone(), q.clone()
    read = [q, k, pos, inv, slots, cu, lens]

    def versions(*x):
        return [t._version for t in x]
    before = versions(*read)
    for call, written in (
            (lambda: msa.msa_rotary(q, k, pos, inv, q_out=qo, k_out=ko), (qo, ko)),
            (lambda: msa.msa_rotary_insert(q, k, k, pos, inv, slots, *caches, q_out=qo, k_out=ko), (qo, ko, *caches)),
            (lambda: msa.msa_rotary_insert(q, k, k, pos, inv, slots, *caches), caches),
            (lambda: (msa.msa_attend_chunk_fp8kv if fp8 else msa.msa_attend_chunk)(q, *caches, lens, table, cu, out=out, lse=lse),
             (out, lse)),
            (lambda: msa.msa_map_slots(lens, lens, table, S.ints([0]), S.ints([1]), num_slots=128, capacity=3), (table,))):
        was = versions(*written)
        call()
        assert all(b > a for a, b in zip(was, versions(*written)))
    assert versions(*read) == before
    with torch.inference_mode():  # tensors without a version
        x = msa.msa_rotary(q.clone(), None, pos, inv, q_out=torch.empty_like(q))[0]
    assert torch.equal(x, msa.msa_rotary(q, None, pos, inv)[0])


def test_slots_of_the_longest_requests():
    # lengths up to 2^31 - 1: a table of 2^24 pages; the pages of an old length next to 2^31
    width = 2 ** 24
    table = torch.full((2, width), 3, dtype=torch.int32, device="cuda")
    longest = 2 ** 31 - 1
    # request 0's token lies in a page that it holds; request 1's open its last page
    lens, news, free = S.ints([longest, longest]), S.ints([1, 200]), S.ints([7, 5])
    ws = msa.Workspace(256)
    cu, slots, positions, left = msa.msa_map_slots(lens, news, table, free, S.ints([2]), num_slots=1024, capacity=201, workspace=ws)
    assert ws.read_device_error() == (0, 0)
    assert cu.tolist() == [0, 1, 201] and int(left) == 1
    at = [longest - 1] + list(range(longest - 200, longest))
    assert positions.tolist() == at
    pages = [3] + [5 if p // 128 == width - 1 else 3 for p in at[1:]]
    assert slots.tolist() == [i * 128 + p % 128 for i, p in zip(pages, at)]
    assert int(table[1, -1]) == 5
    table[1, -1] = 3
    assert bool((table == 3).all())


def test_calls_from_several_threads_at_once():
    # four threads, a stream each, all kinds of calls in turn: each gets the results of calls made one at a time
    def work(seed):
        lens, news = [700 + 300 * seed, 40, 3000], [1 + 5 * seed, 1, 17]
        table, pool = S.page_table(lens, seed=seed)
        gen = torch.Generator("cuda").manual_seed(seed)
        t = sum(news)
        qkv = torch.randn(t, 72, 128, generator=gen, device="cuda").bfloat16()
        dt = torch.float8_e4m3fn if seed % 2 else torch.bfloat16
        k_cache, v_cache = (torch.randn(pool * 128, 4, 128, generator=gen, device="cuda").to(dt) for _ in range(2))
        inv = torch.rand(64, generator=gen, device="cuda")
        out = []
        for _ in range(12):
            cu, slots, pos, left = msa.msa_map_slots(S.ints(lens), S.ints(news), table, S.ints([0]), S.ints([0]),
                                                     num_slots=pool * 128, capacity=t)
            q = msa.msa_rotary_insert(qkv[:, :64], qkv[:, 64:68], qkv[:, 68:], pos, inv, slots, k_cache, v_cache)
            a, b = q[:, :8 + seed].detach().clone().requires_grad_(), qkv[:, 64:65 + seed].detach().clone().requires_grad_()
            y = msa.rotary(a, b, pos, inv)
            out += [cu, slots, pos, left, q, *y, *torch.autograd.grad(y, (a, b), [x * 2 for x in y]),
                    (msa.msa_attend_chunk_fp8kv if seed % 2 else msa.msa_attend_chunk)(q, k_cache, v_cache, S.ints(lens), table, cu)]
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


def test_transforms_that_the_rotation_does_not_have_are_refused():
    pos, inv = S.ints([0, 1, 2]), torch.ones(64, device="cuda")
    x = torch.ones(2, 3, 4, 128, device="cuda").bfloat16()
    with pytest.raises(RuntimeError):
        torch.vmap(lambda a: msa.rotary(a, a, pos, inv)[0])(x)
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises(RuntimeError):
            msa.rotary(torch.autograd.forward_ad.make_dual(x[0], x[1]), x[0], pos, inv)
    assert torch.isfinite(msa.rotary(x[0], x[0], pos, inv)[0]).all()


def test_a_captured_step_refilled_between_replays():
    # a captured serving step whose lengths, tables and positions change between replays, a workspace given by its caller
    lens, news, width, pool = [100, 300], [3, 1], 8, 16
    gen = torch.Generator("cuda").manual_seed(5)
    seq, new = S.ints(lens), S.ints(news)
    table, free = torch.full((2, width), -1, dtype=torch.int32, device="cuda"), torch.randperm(pool, generator=gen, device="cuda").int()
    left = S.ints([pool])
    caches = [torch.full((pool * 128, 4, 128), math.nan, device="cuda").bfloat16() for _ in range(2)]
    cap = 8
    qkv = torch.empty(cap, 72, 128, dtype=torch.bfloat16, device="cuda")
    inv = torch.rand(64, generator=gen, device="cuda")
    ws = msa.Workspace(msa.workspace_size(msa.make_config(), 4, 512, width))

    def step(rows, x):
        cu, slots, pos, now = msa.msa_map_slots(seq, new, table, free, left, num_slots=pool * 128, capacity=rows, workspace=ws)
        q = msa.msa_rotary_insert(x[:, :64], x[:, 64:68], x[:, 68:], pos, inv, slots, *caches, workspace=ws)
        out = msa.msa_attend_chunk(q, *caches, seq, table, cu, workspace=ws)
        left.copy_(now)
        return q, out, cu
    # the prompts, eagerly
    new.copy_(seq)
    step(400, torch.randn(400, 72, 128, generator=gen, device="cuda").bfloat16())
    torch.cuda.synchronize()
    graph, saved = torch.cuda.CUDAGraph(), [x.clone() for x in (left, table)]
    with torch.cuda.graph(graph):
        q, out, cu = step(cap, qkv)
    left.copy_(saved[0]), table.copy_(saved[1])
    for news in ([3, 1], [1, 1], [1, 7], [5, 0], [1, 1]):
        lens = [n + m for n, m in zip(lens, news)]
        seq.copy_(S.ints(lens)), new.copy_(S.ints(news))
        qkv.copy_(torch.randn(cap, 72, 128, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert ws.read_device_error()[0] == 0 and cu.tolist() == S.offsets(news).tolist()
        t = sum(news)
        ref = S.attend(q[:t], *caches, lens, table, cu, SCALE)
        S.check_attend(out[:t], None, ref, max(lens), 8)
