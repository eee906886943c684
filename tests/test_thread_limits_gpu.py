"""Calls of different sizes from two threads, without the interpreter between them: no call's settings of a kernel may refuse
another's launch."""
import ctypes
import subprocess

import pytest
import torch

import block_sparse_attention_08_gb300 as msa
import msa_synth

pytestmark = pytest.mark.gpu

HAMMER = r"""
#include <pthread.h>
#include <stddef.h>
typedef int (*select_t)(const void*, const void*, const void*, const void*, int, long long, int, void*, void*, size_t, void*);
typedef struct { select_t f; const void *cfg, *q, *k, *cu; void *q2k, *ws, *stream; long long tokens; size_t bytes;
                 int docs, longest, times, refused; } call;
static void* work(void* p) {
  call* c = p;
  for (int i = 0; i < c->times; ++i)
    c->refused += c->f(c->cfg, c->q, c->k, c->cu, c->docs, c->tokens, c->longest, c->q2k, c->ws, c->bytes, c->stream) != 0;
  return 0;
}
void hammer(call* c, int n) {
  pthread_t t[8];
  for (int i = 0; i < n; ++i) pthread_create(&t[i], 0, work, &c[i]);
  for (int i = 0; i < n; ++i) pthread_join(t[i], 0);
}
"""


class _Call(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("f", "cfg", "q", "k", "cu", "q2k", "ws", "stream")]
                + [("tokens", ctypes.c_longlong), ("bytes", ctypes.c_size_t)]
                + [(n, ctypes.c_int) for n in ("docs", "longest", "times", "refused")])


def test_prefill_selection_of_short_and_long_documents(tmp_path):
    (tmp_path / "hammer.c").write_text(HAMMER)
    subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-pthread", str(tmp_path / "hammer.c"), "-o", str(tmp_path / "h.so")],
                   check=True)
    hammer = ctypes.CDLL(str(tmp_path / "h.so")).hammer
    lib, cfg = msa.load(), msa.make_config()
    inputs = [msa_synth.prefill_inputs([n], seed=n, device="cuda") for n in (128, 3000)]
    want = [msa.msa_select_blocks_prefill(p.index_q, p.index_k, p.cu_seqlens, p.max_seqlen) for p in inputs]
    calls, kept = (_Call * 2)(), []
    for c, p, w in zip(calls, inputs, want):
        ws = msa.Workspace(msa.workspace_size(cfg, 1, p.total_tokens, -(-p.max_seqlen // 128)))
        out, stream = torch.empty_like(w), torch.cuda.Stream()
        kept.append((ws, out, stream))
        c.f, c.cfg = ctypes.cast(lib.msa_select_blocks_prefill, ctypes.c_void_p).value, ctypes.addressof(cfg)
        c.q, c.k, c.cu, c.q2k = (x.data_ptr() for x in (p.index_q, p.index_k, p.cu_seqlens, out))
        c.ws, c.bytes, c.stream = ws.buf.data_ptr(), ws.nbytes, stream.cuda_stream
        c.tokens, c.docs, c.longest, c.times = p.total_tokens, 1, p.max_seqlen, 400
    torch.cuda.synchronize()
    for _ in range(20):
        hammer(calls, 2)
        torch.cuda.synchronize()
    assert [c.refused for c in calls] == [0, 0]
    assert all(torch.equal(w, out) for w, (_, out, _) in zip(want, kept))


HAMMER_SPARSE = r"""
#include <pthread.h>
#include <stddef.h>
typedef int (*attend_t)(const void*, const void*, const void*, const void*, const void*, const void*, const void*, const void*,
                        const void*, int, int, long long, float, void*, void*, size_t, void*);
typedef struct { attend_t f; const void *cfg, *q, *k, *v, *ks, *vs, *q2k, *lens, *table; void *out, *ws, *stream; long long slots;
                 size_t bytes; float scale; int batch, width, times, refused; } call;
static void* work(void* p) {
  call* c = p;
  for (int i = 0; i < c->times; ++i)
    c->refused += c->f(c->cfg, c->q, c->k, c->v, c->ks, c->vs, c->q2k, c->lens, c->table, c->batch, c->width, c->slots, c->scale,
                       c->out, c->ws, c->bytes, c->stream) != 0;
  return 0;
}
void hammer(call* c, int n) {
  pthread_t t[8];
  for (int i = 0; i < n; ++i) pthread_create(&t[i], 0, work, &c[i]);
  for (int i = 0; i < n; ++i) pthread_join(t[i], 0);
}
"""


class _SparseCall(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("f", "cfg", "q", "k", "v", "ks", "vs", "q2k", "lens", "table", "out", "ws", "stream")]
                + [("slots", ctypes.c_longlong), ("bytes", ctypes.c_size_t), ("scale", ctypes.c_float)]
                + [(n, ctypes.c_int) for n in ("batch", "width", "times", "refused")])


@pytest.mark.parametrize("batches", [(4, 64), (1, 9, 10, 20)])
def test_sparse_attention_of_few_and_many_requests_over_an_int8_cache(batches, tmp_path):
    """Few requests' CTAs take an SM each, many share one: the launches ask for different amounts of shared memory."""
    (tmp_path / "hammer.c").write_text(HAMMER_SPARSE)
    subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-pthread", str(tmp_path / "hammer.c"), "-o", str(tmp_path / "h.so")],
                   check=True)
    hammer = ctypes.CDLL(str(tmp_path / "h.so")).hammer
    lib, cfg = msa.load(), msa.make_config()
    gen = torch.Generator("cuda").manual_seed(1)
    pages, width = 64, 16
    k, v = (torch.randint(-127, 128, (pages * 128, 4, 128), generator=gen, device="cuda", dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(-7, -4, (pages, 4, 128), generator=gen, device="cuda").float()).bfloat16() for _ in range(2))
    calls, kept = (_SparseCall * len(batches))(), []
    for c, n in zip(calls, batches):
        q = torch.randn(n, 64, 128, generator=gen, device="cuda").bfloat16()
        table = torch.randint(0, pages, (n, width), generator=gen, device="cuda", dtype=torch.int32)
        lens = torch.full((n,), width * 128 - 5, dtype=torch.int32, device="cuda")
        q2k = torch.arange(width, dtype=torch.int32, device="cuda").expand(4, n, width).contiguous()
        want = msa.msa_sparse_attend_decode_int8kv(q, k, v, ks, vs, q2k, lens, table)
        ws, out, stream = msa.Workspace(256), torch.empty_like(want), torch.cuda.Stream()
        kept.append((q, table, lens, q2k, want, ws, out, stream))
        c.f, c.cfg = ctypes.cast(lib.msa_sparse_attend_decode_int8kv, ctypes.c_void_p).value, ctypes.addressof(cfg)
        c.q, c.k, c.v, c.ks, c.vs, c.q2k, c.lens, c.table, c.out = (
            x.data_ptr() for x in (q, k, v, ks, vs, q2k, lens, table, out))
        c.ws, c.bytes, c.stream = ws.buf.data_ptr(), ws.nbytes, stream.cuda_stream
        c.slots, c.scale, c.batch, c.width, c.times = pages * 128, 128 ** -0.5, n, width, 400
    torch.cuda.synchronize()
    for _ in range(20):
        hammer(calls, len(batches))
        torch.cuda.synchronize()
    assert [c.refused for c in calls] == [0] * len(batches)
    for _, _, _, _, want, ws, out, _ in kept:
        assert ws.read_device_error() == (0, 0) and torch.equal(want, out)
