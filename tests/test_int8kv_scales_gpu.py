"""Every kind of scale in an int8 cache, through each attention: one key takes all of a row's weight, so the output is that key's
value, exactly; and a token that sees one key has that key's score as its log-sum-exp."""
import math

import pytest
import torch

import _serving as S
import block_sparse_attention_08_gb300 as msa

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(128.0)


def _v_scales(kind):
    """128 scales: powers of two down to the smallest (a row of zeros has that), or any, among them zeros and negative ones."""
    if kind == "powers":
        return torch.tensor([2.0 ** e for e in range(-133, 120, 2)] + [2.0 ** 119], dtype=torch.float64)
    if kind == "large powers":  # (128 and 256 times such a scale are no bf16 numbers)
        return torch.tensor([2.0 ** (e % 20 + 102) for e in range(128)], dtype=torch.float64)
    gen = torch.Generator().manual_seed(1)
    s = torch.exp2(torch.rand(128, generator=gen, dtype=torch.float64) * 100 - 50).bfloat16().double()
    s[::5] *= -1
    s[3], s[40], s[77] = 0.0, -0.0, 3 * 2.0 ** -133
    s[64:80] = 2.0 ** -6
    return s


def _one_key_each(kind):
    """Two pages: key i < 128 is 127 in dim i, the others zero; row (token, head h) asks for key (16 token + h % 16) % 128."""
    k = torch.zeros(256, 4, 128, dtype=torch.int8)
    k[torch.arange(128), :, torch.arange(128)] = 127
    v = torch.randint(-127, 128, (256, 4, 128), generator=torch.Generator().manual_seed(2), dtype=torch.int32).to(torch.int8)
    ks = torch.ones(2, 4, 128, dtype=torch.bfloat16)
    vs = torch.ones(2, 4, 128, dtype=torch.bfloat16)
    s = _v_scales(kind)
    for g in range(4):
        vs[0, g] = s.roll(31 * g).bfloat16()
    return [x.cuda() for x in (k, v, ks, vs)]


def _ask(tokens, first=0):
    q = torch.zeros(tokens, 64, 128)
    key = (16 * (torch.arange(tokens)[:, None] + first) + torch.arange(64)[None] % 16) % 128
    q.scatter_(2, key[..., None], 40.0)
    return q.bfloat16().cuda(), key.cuda()


def _check(out, key, v, vs):
    g = (torch.arange(64, device="cuda") // 16).expand(key.shape)
    want = (v[key, g].double() * vs[0][g, key].double()[..., None]).bfloat16().double()
    # fp32 sums of values below its normal numbers may be lost
    assert bool(((out.double() - want).abs() <= 2.0 ** -126).all())
    normal = want.abs() >= 2.0 ** -126
    assert torch.equal(out.double()[normal], want[normal])


@pytest.mark.parametrize("kind", ["powers", "large powers", "any"])
def test_values(kind):
    k, v, ks, vs = _one_key_each(kind)
    table = S.ints([[0, 1]])
    for n in (16, 5, 2):
        q, key = _ask(n)
        _check(msa.msa_attend_chunk_int8kv(q, k, v, ks, vs, S.ints([128 + n]), table, S.offsets([n])), key, v, vs)
    tables = table.expand(8, 2).contiguous()
    q, key = _ask(8)
    lens = S.ints([129 + 3 * i for i in range(8)])
    cu = S.offsets([1] * 8)
    _check(msa.msa_attend_shared_int8kv(q, k, v, ks, vs, lens, tables, cu, S.ints([0, 8]), S.ints([128])), key, v, vs)
    # One token's warps take 32 keys each, and most of them have none but such that score zero: 32 weights of 1 times values of up
    # to 2^128 are no fp32 sum.
    if kind != "large powers":
        _check(msa.msa_attend_chunk_int8kv(q, k, v, ks, vs, lens, tables, cu), key, v, vs)
        q2k = S.ints([[[0, 1]] * 8] * 4)
        _check(msa.msa_sparse_attend_decode_int8kv(q, k, v, ks, vs, q2k, lens, tables), key, v, vs)
    got = msa.msa_dequantize_gather(k, v, ks, vs, table, S.ints([0, 128]), 128)[1]
    want = (v[:128].double() * vs[0].T.double()[..., None]).bfloat16()
    assert torch.equal(got.double(), want.double())


@pytest.mark.parametrize("tokens", [1, 2])
def test_scores(tokens):
    # 1.5: no power of two; 2^120, 2^121: none that is put under the bits
    scales = [2.0 ** e for e in range(-118, 119, 4)] + [1.5 * 2.0 ** e for e in range(-118, 119, 7)] + [-1.0, 2.0 ** 119, 2.0 ** 120]
    n = len(scales)
    k = torch.zeros(n * 128, 4, 128, dtype=torch.int8)
    k[::128] = torch.randint(-127, 128, (n, 4, 128), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(torch.int8)
    ks = torch.ones(n, 4, 128, dtype=torch.bfloat16)
    ks[:, :, 0] = torch.tensor(scales).bfloat16()[:, None]
    k, ks = k.cuda(), ks.cuda()
    v, vs = torch.zeros_like(k), torch.ones_like(ks)
    q = torch.zeros(n * tokens, 64, 128, dtype=torch.float64)
    q[::tokens] = torch.randn(n, 64, 128, generator=torch.Generator().manual_seed(4), dtype=torch.float64) / 64
    q[::tokens] /= torch.tensor(scales, dtype=torch.float64)[:, None, None]
    q = q.bfloat16().cuda()
    lse = torch.empty(n * tokens, 64, device="cuda")
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
    msa.msa_attend_chunk_int8kv(q, k, v, ks, vs, S.ints([tokens] * n), table, S.offsets([tokens] * n), lse=lse)
    value = (k[::128].double() * ks[:, :, 0].double()[..., None]).bfloat16().double()  # [n, 4, 128]
    if tokens == 1:
        value = k[::128].double() * ks[:, :, 0].double()[..., None]  # (the scale multiplies the score)
    x = q[::tokens].double() * value.repeat_interleave(16, 1) * SCALE
    want, reach = x.sum(-1) / math.log(2.0), x.abs().sum(-1)
    # 128 sums of products in fp32, and the factors; the logarithm of one weight is zero
    tol = 1.4427 * reach * 132 * 2.0 ** -24 + 2.0 ** -20
    assert bool(((lse[::tokens].double() - want).abs() <= tol).all())
