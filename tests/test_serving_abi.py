"""Refusals of the chunked-serving calls, without a GPU: nothing is enqueued and no pointer is read."""
import ctypes
import math

import pytest
import torch

import block_sparse_attention_08_gb300 as msa
from block_sparse_attention_08_gb300.binding import msa_config, msa_rotary_config

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


def test_map_slots(lib):
    good = [FAKE, FAKE, 4, FAKE, 8, FAKE, 100, FAKE, 1280, 50, FAKE, FAKE, FAKE, 2 * FAKE, FAKE, 256, None]
    _refuses(lib.msa_map_slots, good, [
        (0, None, NULL), (1, None, NULL), (2, 0, SHAPE), (3, None, NULL), (4, 0, SHAPE), (5, None, NULL), (6, -1, SHAPE),
        (6, 1 << 31, SHAPE), (7, None, NULL), (8, 0, SHAPE), (8, 1000, SHAPE), (8, 1 << 31, SHAPE), (9, 0, SHAPE),
        (9, 1 << 31, SHAPE), (10, None, NULL), (11, None, NULL), (12, None, NULL), (13, None, NULL), (13, FAKE, SHAPE),
        (14, None, WORKSPACE), (14, FAKE + 8, WORKSPACE), (15, 255, WORKSPACE)])


def _rot(rot_dim=128, interleaved=0, num_axes=3, axis=None):
    c = msa_rotary_config(rot_dim, interleaved, num_axes)
    for j, a in enumerate(axis or []):
        c.axis[j] = a
    return ctypes.byref(c)


BAD_ROT = [(None, NULL), (_rot(0), SHAPE), (_rot(8), SHAPE), (_rot(24), SHAPE), (_rot(144), SHAPE), (_rot(interleaved=2), SHAPE),
           (_rot(num_axes=0), SHAPE), (_rot(num_axes=5), SHAPE), (_rot(axis=[0] * 63 + [3]), SHAPE)]


def test_rotary(lib):
    good = [_rot(), FAKE, 8192, 64, FAKE, 512, 4, FAKE, FAKE, 10, 0, FAKE, FAKE, None]
    _refuses(lib.msa_rotary, good, [(0, c, code) for c, code in BAD_ROT] + [
        (1, None, NULL), (1, FAKE + 8, ALIGN), (2, 8191, SHAPE), (2, 8196, SHAPE), (2, 8184, SHAPE), (3, 0, SHAPE), (3, 65, SHAPE),
        (4, None, NULL), (4, FAKE + 2, ALIGN), (5, 511, SHAPE), (5, 504, SHAPE), (6, 0, SHAPE), (6, 65, SHAPE), (7, None, NULL),
        (8, None, NULL), (9, 0, SHAPE), (9, 1 << 31, SHAPE), (11, None, NULL), (11, FAKE + 4, ALIGN), (12, None, NULL),
        (12, FAKE + 4, ALIGN)])


def test_rotary_insert(lib):
    good = [_rot(), FAKE, 9216, FAKE, 9216, FAKE, 9216, FAKE, FAKE, FAKE, 10, FAKE, None, FAKE, FAKE, 1, 1.0, 1.0, 1280, FAKE,
            256, None]
    nan, inf = math.nan, math.inf
    _refuses(lib.msa_rotary_insert, good, [(0, c, code) for c, code in BAD_ROT] + [
        (1, None, NULL), (2, 9217, SHAPE), (3, None, NULL), (3, FAKE + 2, ALIGN), (4, 504, SHAPE), (4, 513, SHAPE), (5, None, NULL),
        (5, FAKE + 2, ALIGN), (6, 504, SHAPE), (7, None, NULL), (8, None, NULL), (9, None, NULL), (10, 0, SHAPE), (11, None, NULL),
        (12, FAKE + 2, ALIGN), (13, None, NULL), (13, FAKE + 2, ALIGN), (14, None, NULL), (14, FAKE + 2, ALIGN), (16, 0.0, SHAPE),
        (16, nan, SHAPE), (17, inf, SHAPE), (17, -1.0, SHAPE), (18, 0, SHAPE), (18, 1 << 31, SHAPE), (19, None, WORKSPACE),
        (20, 100, WORKSPACE)])


def test_attend_chunk(lib):
    cfg, size = msa_config(), ctypes.c_size_t()
    assert lib.msa_config_default(ctypes.byref(cfg)) == OK
    assert lib.msa_workspace_size(ctypes.byref(cfg), 4, 100, 9, ctypes.byref(size)) == OK and size.value >= 256
    bad = msa_config()
    lib.msa_config_default(ctypes.byref(bad))
    bad.head_dim = 64
    good = [ctypes.byref(cfg), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 9, 100, 1280, 0.1, FAKE, None, FAKE, size.value, None]
    cases = [(0, None, NULL), (0, ctypes.byref(bad), SHAPE), (1, None, NULL), (1, FAKE + 8, ALIGN), (2, None, NULL),
             (2, FAKE + 8, ALIGN), (3, None, NULL), (3, FAKE + 8, ALIGN), (4, None, NULL), (5, None, NULL), (6, None, NULL),
             (7, 0, SHAPE), (8, 0, SHAPE), (8, 1 << 24, SHAPE), (9, 0, SHAPE), (9, 1 << 31, SHAPE), (10, 0, SHAPE), (10, 1000, SHAPE),
             (10, 1 << 31, SHAPE), (11, 0.0, SHAPE), (11, -1.0, SHAPE), (11, math.nan, SHAPE), (11, math.inf, SHAPE),
             (12, None, NULL), (12, FAKE + 8, ALIGN), (14, None, WORKSPACE), (14, FAKE + 16, WORKSPACE),
             (15, size.value - 1, WORKSPACE)]
    _refuses(lib.msa_attend_chunk, good, cases)
    fp8 = good[:4] + [1.0, 1.0] + good[4:]
    _refuses(lib.msa_attend_chunk_fp8kv, fp8, [(w if w < 4 else w + 2, v, c) for w, v, c in cases] + [
        (4, 0.0, SHAPE), (4, math.nan, SHAPE), (5, -1.0, SHAPE), (5, math.inf, SHAPE)])


def test_the_binding_refuses_other_tensors():
    x = torch.zeros(4, 64, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        msa.msa_attend_chunk(x, x, x, i, i[None], i)
    with pytest.raises(ValueError, match="q has shape .4,., expected 3 dimensions"):
        msa.msa_attend_chunk(i, x, x, i, i, i)
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        msa.msa_attend_chunk_fp8kv(None, x, x, i, i[None], i)
    with pytest.raises(ValueError, match="CUDA"):
        msa.msa_rotary(x, None, i, torch.zeros(64))
    with pytest.raises(ValueError, match="axes has 3 entries, inv_freq has 64"):
        msa.msa_rotary(x, None, i, torch.zeros(64), axes=(0, 0, 0))
    with pytest.raises(ValueError, match="axes must lie"):
        msa.msa_rotary(x, None, i, torch.zeros(2), axes=[0, 1])
    with pytest.raises(ValueError, match="at most 64 pairs"):
        msa.msa_rotary(x, None, i, torch.zeros(65))
    with pytest.raises(TypeError):
        msa.msa_rotary(x, None, i, torch.zeros(2), axes=[0, "x"])
    with pytest.raises(TypeError):
        msa.msa_rotary_insert(x, x, x, i, torch.zeros(64), i, x, x, k_scale="x")
    with pytest.raises(ValueError, match="CUDA"):
        msa.msa_map_slots(i, i, i[None], i, i[:1], num_slots=128, capacity=1)
    with pytest.raises(TypeError):
        msa.msa_map_slots(i, i, i[None], i, i[:1], num_slots=128, capacity=1.5)
