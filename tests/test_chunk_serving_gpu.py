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


def test_refusals_of_wrong_tensors():
    def ints(*shape):
        return torch.zeros(shape, dtype=torch.int32, device="cuda")
    q = torch.zeros(4, 64, 128, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(256, 4, 128, dtype=torch.bfloat16, device="cuda")
    freq, slots = torch.ones(64, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    attend = [q, c, c, ints(2), ints(2, 3), ints(3)]
    for where, bad, text in ((0, q.float(), "dtype"), (0, q[:, ::2], "shape"), (0, q.transpose(0, 1)[:4], "shape|contiguous"),
                             (0, q.repeat(2, 1, 1)[::2], "contiguous"), (1, c[:, :2], "shape"), (1, c.half(), "k_cache must be bf16"),
                             (2, c[:128], "shape"), (2, c.to(torch.float8_e4m3fn), "dtype"), (3, ints(3), "shape"),
                             (3, ints(2).long(), "dtype"), (3, ints(2).cpu(), "CUDA"), (4, ints(2, 6)[:, ::2], "contiguous"),
                             (4, ints(2), "dimensions"), (5, ints(2), "shape")):
        args = list(attend)
        args[where] = bad
        with pytest.raises(ValueError, match=text):
            msa.msa_attend_chunk(*args)
    with pytest.raises(ValueError, match="takes float8_e4m3fn or uint8 caches"):
        msa.msa_attend_chunk_fp8kv(*attend)
    with pytest.raises(ValueError, match="takes bf16 caches"):
        msa.msa_attend_chunk(q, c.to(torch.float8_e4m3fn), c.to(torch.float8_e4m3fn), *attend[3:])
    with pytest.raises(ValueError, match="lse"):
        msa.msa_attend_chunk(*attend, lse=torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="out"):
        msa.msa_attend_chunk(*attend, out=q[:3])
    for kw in ({"scale": 0.0}, {"scale": math.nan}, {"workspace": msa.Workspace(256)}):
        with pytest.raises(msa.MsaError):
            msa.msa_attend_chunk(*attend, **kw)
    with pytest.raises(msa.MsaError):  # no rows
        msa.msa_attend_chunk(q[:0], *attend[1:])
    k, pos = q[:, :4].contiguous(), ints(4)
    for args, text in (((q, k, ints(5), freq), "positions"), ((q, k[:3], pos, freq), "k has shape"),
                       ((q[:, :, ::2], k, pos, freq), "q has shape"), ((q[..., :64].repeat(1, 1, 2)[:, ::2], k, pos, freq), "dense heads"),
                       ((q, k, pos, freq.double()), "inv_freq")):
        with pytest.raises(ValueError, match=text):
            msa.msa_rotary(*args)
    with pytest.raises(ValueError, match="tokens"):
        msa.msa_rotary(q[:1].expand(4, 64, 128), None, pos, freq)
    with pytest.raises(ValueError, match="k_out without k"):
        msa.msa_rotary(q, None, pos, freq, k_out=k)
    with pytest.raises(msa.MsaError):  # 12 pairs: rot_dim 24
        msa.msa_rotary(q, None, pos, freq[:12].contiguous())
    insert = [q, k, k, pos, freq, slots, c, c]
    for where, bad, text in ((2, k.float(), "v must have dtype"), (5, slots.int(), "slots"), (6, c[:, :3], "k_cache"),
                             (7, c.to(torch.float8_e4m3fn), "v_cache")):
        args = list(insert)
        args[where] = bad
        with pytest.raises(ValueError, match=text):
            msa.msa_rotary_insert(*args)
    b8 = c.to(torch.float8_e4m3fn)
    with pytest.raises(msa.MsaError):
        msa.msa_rotary_insert(*insert[:6], b8, b8, k_scale=-1.0)
    slot_args = [ints(2), ints(2), ints(2, 3), ints(5), ints(1)]
    for kw in ({"num_slots": 100, "capacity": 4}, {"num_slots": 128, "capacity": 0},
               {"num_slots": 128, "capacity": 4, "num_free_out": slot_args[4]}):
        with pytest.raises(msa.MsaError):
            msa.msa_map_slots(*slot_args, **kw)
    with pytest.raises(ValueError, match="new_lens"):
        msa.msa_map_slots(slot_args[0], ints(3), *slot_args[2:], num_slots=128, capacity=4)


@pytest.mark.parametrize("fp8", [False, True])
def test_one_workspace_for_chunks_and_the_sparse_decode(fp8):
    """A step of chunks between two decode steps leaves the decode calls' counters in a shared workspace alone."""
    gen = torch.Generator("cuda").manual_seed(3)
    lens = [5000, 700, 3000, 129]
    table, pool = S.page_table(lens)
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    k, v = (torch.randn(pool * 128, 4, 128, generator=gen, device="cuda").to(dt) for _ in range(2))
    index = torch.randn(pool * 128, 1, 128, generator=gen, device="cuda").bfloat16()
    iq = torch.randn(4, 4, 128, generator=gen, device="cuda").bfloat16()
    q = torch.randn(4, 64, 128, generator=gen, device="cuda").bfloat16()
    news = [40, 1, 17, 8]
    qc = torch.randn(sum(news), 64, 128, generator=gen, device="cuda").bfloat16()
    cfg, width = msa.make_config(), table.shape[1]
    ws = msa.Workspace(max(msa.workspace_size(cfg, 0, 4, width), msa.workspace_size(cfg, 4, sum(news), width)))
    decode = msa.msa_sparse_attend_decode_fp8kv if fp8 else msa.msa_sparse_attend_decode
    chunk = msa.msa_attend_chunk_fp8kv if fp8 else msa.msa_attend_chunk

    def steps(workspace):
        out = []
        for i in range(3):
            q2k = msa.msa_select_blocks_decode(iq, index, S.ints(lens), page_table=table, workspace=workspace)
            out += [q2k, decode(q, k, v, q2k, S.ints(lens), page_table=table, workspace=workspace)]
            out.append(chunk(qc, k, v, S.ints(lens), table, S.offsets(news), workspace=workspace))
            out.append(chunk(qc[:4], k, v, S.ints(lens), table, S.offsets([1] * 4), workspace=workspace))
        return out
    shared = steps(ws)
    assert ws.read_device_error()[0] == 0
    for i, (a, b) in enumerate(zip(shared[:8] + shared, shared[4:] + steps(None))):
        if i % 4 == 1:
            # the decode attention may join its pieces in another order: one bf16 step, and fp32 sums of values below 8
            assert bool(((a.float() - b.float()).abs() <= 2.0 ** -7 * a.float().abs() + 2.0 ** -16).all())
        else:
            assert torch.equal(a, b)
