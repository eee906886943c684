"""Calls of the chunk-serving functions at the borders of what they accept: addresses, threads, frequencies, lengths,
buffers that change behind autograd."""
import math

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
