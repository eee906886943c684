"""Borders of the chunk-serving calls that need no GPU."""
import ctypes

import pytest

import block_sparse_attention_08_gb300 as msa
from block_sparse_attention_08_gb300.binding import msa_config

OK, NULL, SHAPE, DTYPE, WORKSPACE, ALIGN = 0, 1, 2, 3, 4, 5
FAKE = 0x10000  # 256-byte aligned, never read: every call below is refused first


@pytest.fixture(scope="module")
def lib():
    return msa.load()


def test_a_score_factor_that_is_no_normal_number_is_refused(lib):
    # scale and k_scale are finite and positive, scale * log2(e) * k_scale is not, or subnormal.  An accepted factor is
    # refused for its workspace instead, so that nothing runs.
    cfg = msa_config()
    lib.msa_config_default(ctypes.byref(cfg))
    tail = [FAKE, FAKE, FAKE, 4, 9, 100, 1280]
    for scale, code in ((3e38, SHAPE), (2.4e38, SHAPE), (2.3e38, WORKSPACE), (1e-39, SHAPE), (8e-39, SHAPE), (1e-38, WORKSPACE),
                        (0.088, WORKSPACE)):
        assert lib.msa_attend_chunk(ctypes.byref(cfg), FAKE, FAKE, FAKE, *tail, scale, FAKE, None, FAKE, 0, None) == code, scale
    for scale, k_scale, code in ((1e-30, 1e-30, SHAPE), (1e30, 1e30, SHAPE), (1e30, 1e-30, WORKSPACE), (1e-30, 1e30, WORKSPACE),
                                 (0.088, 1e-38, SHAPE), (0.088, 3e38, WORKSPACE), (10.0, 3e38, SHAPE)):
        assert lib.msa_attend_chunk_fp8kv(ctypes.byref(cfg), FAKE, FAKE, FAKE, k_scale, 1.0, *tail, scale, FAKE, None, FAKE, 0,
                                          None) == code, (scale, k_scale)
