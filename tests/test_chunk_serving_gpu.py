"""A serving loop over the paged cache: pages, rotation, insertion and attention, as a program calls them."""
import math

import pytest
import torch

import _serving as S
import block_sparse_attention_08_gb300 as msa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_prompts_in_chunks_then_single_tokens(fp8):
    """Three requests' prompts arrive in chunks, then each decodes: every step's attention is compared with
    the 64-bit attention over the keys that the steps so far have inserted, kept apart by the test."""
    gen = torch.Generator("cuda").manual_seed(1)
    B, width, pool, rot = 3, 6, 20, 64
    axes = tuple([0] * 12 + [1] * 10 + [2] * 10)
    inv_freq = torch.tensor([1e4 ** (-2.0 * j / rot) for j in range(rot // 2)], device="cuda")
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    scales = {"k_scale": 0.05, "v_scale": 0.03} if fp8 else {}
    k_cache = torch.full((pool * 128, 4, 128), math.nan, device="cuda").to(dt)
    v_cache = k_cache.clone()
    index_cache = torch.zeros(pool * 128, 1, 128, dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pool, generator=gen, device="cuda", dtype=torch.int32)
    left = S.ints([pool])
    lens = [0] * B
    seen = [[] for _ in range(B)]  # slot of each position
    ws = msa.Workspace(msa.workspace_size(msa.make_config(), 4, 512, width))
    for news in ([130, 7, 0], [128, 1, 300], [1, 100, 129], [1, 1, 1], [1, 0, 1], [1, 1, 1]):
        lens = [n + m for n, m in zip(lens, news)]
        cap = sum(news) + 3
        cu, slots, positions, left = msa.msa_map_slots(S.ints(lens), S.ints(news), table, free, left,
                                                       num_slots=pool * 128, capacity=cap, workspace=ws)
        qkv = torch.randn(cap, 72, 128, generator=gen, device="cuda").bfloat16()
        q, k, v = qkv[:, :64], qkv[:, 64:68], qkv[:, 68:]
        pos3 = torch.stack([positions, positions // 3, positions % 7])
        ko = torch.empty(cap, 4, 128, dtype=torch.bfloat16, device="cuda")
        qr = msa.msa_rotary_insert(q, k, v, pos3, inv_freq, slots, k_cache, v_cache, axes=axes, k_out=ko, workspace=ws,
                                   **scales)
        lse = torch.empty(cap, 64, device="cuda")
        call = msa.msa_attend_chunk_fp8kv if fp8 else msa.msa_attend_chunk
        out = call(qr, k_cache, v_cache, S.ints(lens), table, cu, lse=lse, workspace=ws, **scales)
        assert ws.read_device_error()[0] == 0
        total = sum(news)
        assert cu.tolist() == S.offsets(news).tolist() and int(left) == pool - sum(S.pages(n) for n in lens)
        at = 0
        for r, m in enumerate(news):
            seen[r] += slots[at:at + m].tolist()
            at += m
        every = [s for x in seen for s in x]
        assert len(set(every)) == len(every) and min(every) >= 0
        want = S.rotate(k[:total], pos3[:, :total], inv_freq, axes, False)
        got = k_cache[slots[:total]].double() * scales.get("k_scale", 1.0)
        # bf16: 2^-8 of the value; E4M3: 2^-4, or half its smallest step times the scale; and the fp32 rotation
        tol = (2.0 ** -4 if fp8 else 2.0 ** -8) * want.abs() + scales.get("k_scale", 0.0) * 2.0 ** -10 + 2.0 ** -17
        assert bool(((got - want).abs() <= tol).all())
        ref = S.attend(qr[:total], k_cache, v_cache, lens, table, cu, 1 / math.sqrt(128.0), **scales)
        S.check_attend(out[:total], lse[:total], ref, max(lens), 11 if fp8 else 8)
    # the sparse decode over the cache that these calls filled: contexts of at most 16 blocks keep them all
    # (that call gives the masked slots' V the weight zero, so they have to be finite: only the chunk attention reads
    # past NaN there)
    finite = [x.float().nan_to_num(0.0).to(dt) for x in (k_cache, v_cache)]
    iq = torch.randn(B, 4, 128, generator=gen, device="cuda").bfloat16()
    qd = torch.randn(B, 64, 128, generator=gen, device="cuda").bfloat16()
    q2k = msa.msa_select_blocks_decode(iq, index_cache, S.ints(lens), page_table=table.clamp(min=0))
    sparse = (msa.msa_sparse_attend_decode_fp8kv if fp8 else msa.msa_sparse_attend_decode)(
        qd, *finite, q2k, S.ints(lens), page_table=table.clamp(min=0), **scales)
    cu = S.offsets([1] * B)
    ref = S.attend(qd, k_cache, v_cache, lens, table, cu, 1 / math.sqrt(128.0), **scales)
    call = msa.msa_attend_chunk_fp8kv if fp8 else msa.msa_attend_chunk
    S.check_attend(call(qd, k_cache, v_cache, S.ints(lens), table, cu, **scales), None, ref, max(lens), 11 if fp8 else 8)
    S.check_attend(sparse, None, ref, max(lens), 11 if fp8 else 8)
