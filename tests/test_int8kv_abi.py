"""Refusals of the int8-cache calls, without a GPU: nothing is enqueued and no pointer is read."""
import ctypes
import math

import pytest
import torch

import block_sparse_attention_08_gb300 as msa
from block_sparse_attention_08_gb300.binding import msa_config

OK, NULL, SHAPE, DTYPE, WORKSPACE, ALIGN = 0, 1, 2, 3, 4, 5
FAKE = 0x10000  # 256-byte aligned, never read: every call below is refused first


@pytest.fixture(scope="module")
def lib():
    return msa.load()


def _refuses(f, good, cases):
    for where, value, code in cases:
        args = list(good)
        args[where] = value
        assert f(*args) == code, (where, value)


def _tensors(*at):
    return [c for i in at for c in ((i, None, NULL), (i, FAKE + 8, ALIGN))]


def test_quantize_insert(lib):
    good = [FAKE, 512, FAKE, 1024, FAKE, 10, FAKE, FAKE, FAKE, FAKE, 1280, FAKE, 256, None]
    _refuses(lib.msa_quantize_insert, good, _tensors(0, 2, 6, 7, 8, 9) + [
        (1, 504, SHAPE), (1, 516, SHAPE), (3, 511, SHAPE), (3, 1028, SHAPE), (4, None, NULL), (5, 0, SHAPE), (5, 1 << 31, SHAPE),
        (10, 0, SHAPE), (10, 1000, SHAPE), (10, 1 << 31, SHAPE), (11, None, WORKSPACE), (11, FAKE + 8, WORKSPACE),
        (12, 255, WORKSPACE)])


def test_dequantize_gather(lib):
    good = [FAKE, FAKE, FAKE, FAKE, 1280, FAKE, None, FAKE, 4, 9, 100, FAKE, FAKE, FAKE, 256, None]
    _refuses(lib.msa_dequantize_gather, good, _tensors(0, 1, 2, 3, 11, 12) + [
        (4, 0, SHAPE), (4, 1000, SHAPE), (4, 1 << 31, SHAPE), (5, None, NULL), (7, None, NULL), (8, 0, SHAPE), (9, 0, SHAPE),
        (9, 1 << 24, SHAPE), (10, 0, SHAPE), (10, 1 << 31, SHAPE), (13, None, WORKSPACE), (13, FAKE + 8, WORKSPACE),
        (14, 255, WORKSPACE)])


def test_sparse_attend(lib):
    cfg = msa_config()
    assert lib.msa_config_default(ctypes.byref(cfg)) == OK
    good = [ctypes.byref(cfg), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 9, 1280, 0.1, FAKE, FAKE, 256, None]
    _refuses(lib.msa_sparse_attend_decode_int8kv, good, _tensors(1, 2, 3, 4, 5, 13) + [
        (0, None, NULL), (6, None, NULL), (7, None, NULL), (8, None, NULL), (9, 0, SHAPE), (9, 1 << 30, SHAPE), (10, 0, SHAPE), (11, 0, SHAPE),
        (11, 1000, SHAPE), (11, 1 << 31, SHAPE), (12, 0.0, SHAPE), (12, -1.0, SHAPE), (12, math.nan, SHAPE),
        (12, math.inf, SHAPE), (12, 5e-39, SHAPE), (14, None, WORKSPACE), (14, FAKE + 8, WORKSPACE),
        (15, 255, WORKSPACE)])


def test_attend_chunk_and_shared(lib):
    cfg, size, more = msa_config(), ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.msa_config_default(ctypes.byref(cfg)) == OK
    assert lib.msa_workspace_size(ctypes.byref(cfg), 4, 100, 9, ctypes.byref(size)) == OK
    assert lib.msa_workspace_size(ctypes.byref(cfg), 5, 100, 9, ctypes.byref(more)) == OK and more.value > size.value
    bad = msa_config()
    lib.msa_config_default(ctypes.byref(bad))
    bad.head_dim = 64
    c = ctypes.byref(cfg)
    # cfg, q, caches, (scales,) seq_lens, page_table, cu, batch, max_blocks, (groups,) tokens, slots, scale, out, lse, workspace
    for f, head, group in ((lib.msa_attend_chunk_int8kv, [FAKE] * 2, False), (lib.msa_attend_shared, [], True),
                           (lib.msa_attend_shared_fp8kv, [1.0, 1.0], True), (lib.msa_attend_shared_int8kv, [FAKE] * 2, True)):
        groups = [FAKE, FAKE, 2] if group else []
        need = more.value if group else size.value
        good = [c, FAKE, FAKE, FAKE] + head + [FAKE, FAKE, FAKE, 4, 9] + groups + [100, 1280, 0.1, FAKE, None, FAKE, need, None]
        a = 4 + len(head)       # seq_lens
        b = a + 5 + len(groups)  # tokens
        cases = _tensors(1, 2, 3, b + 3) + [
            (0, None, NULL), (0, ctypes.byref(bad), SHAPE), (a, None, NULL), (a + 1, None, NULL), (a + 2, None, NULL), (a + 3, 0, SHAPE),
            (a + 4, 0, SHAPE), (a + 4, 1 << 24, SHAPE), (b, 0, SHAPE), (b, 1 << 31, SHAPE), (b + 1, 0, SHAPE), (b + 1, 1000, SHAPE),
            (b + 1, 1 << 31, SHAPE), (b + 2, 0.0, SHAPE), (b + 2, math.nan, SHAPE), (b + 2, math.inf, SHAPE), (b + 2, -1.0, SHAPE),
            (b + 5, None, WORKSPACE), (b + 5, FAKE + 16, WORKSPACE), (b + 6, need - 1, WORKSPACE)]
        if group:
            cases += [(a + 5, None, NULL), (a + 6, None, NULL), (a + 7, -1, SHAPE), (a + 7, 5, SHAPE), (a + 3, 0x7fffffff, SHAPE)]
        if head == [FAKE] * 2:
            cases += _tensors(4, 5)
        elif head:
            cases += [(4, 0.0, SHAPE), (4, math.nan, SHAPE), (5, -1.0, SHAPE), (5, math.inf, SHAPE), (5, 2.0 ** -81, SHAPE)]
        _refuses(f, good, cases)


def test_the_binding_refuses_other_tensors():
    x = torch.zeros(4, 4, 128, dtype=torch.bfloat16)
    c = torch.zeros(128, 4, 128, dtype=torch.int8)
    s = torch.zeros(1, 4, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="k must be a CUDA tensor"):
        msa.msa_quantize_insert(x, x, i.long(), c, c, s, s)
    with pytest.raises(TypeError, match="v must be a torch.Tensor"):
        msa.msa_quantize_insert(x, None, i.long(), c, c, s, s)
    with pytest.raises(ValueError, match="k has shape .4,., expected 3 dimensions"):
        msa.msa_quantize_insert(i, x, i.long(), c, c, s, s)
    with pytest.raises(ValueError, match="k_cache must be a CUDA tensor"):
        msa.msa_dequantize_gather(c, c, s, s, i[None], i, 4)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        msa.msa_sparse_attend_decode_int8kv(x, c, c, s, s, i[None, None], i, i[None])
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        msa.msa_attend_shared(x, c, c, i, i[None], i, i, i)
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        msa.msa_attend_shared_fp8kv(None, c, c, i, i[None], i, i, i)
    with pytest.raises(ValueError, match="q has shape .4,., expected 3 dimensions"):
        msa.msa_attend_shared_int8kv(i, c, c, s, s, i, i[None], i, i, i)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        msa.msa_attend_chunk_int8kv(x, c, c, s, s, i, i[None], i)
