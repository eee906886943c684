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
