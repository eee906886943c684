"""Borders of the chunk-serving calls that need no GPU."""
import ctypes
import os
import re
import subprocess
import sys
import sysconfig

import pytest
import torch

import block_sparse_attention_08_gb300 as msa
from block_sparse_attention_08_gb300 import _build, binding
from block_sparse_attention_08_gb300.binding import msa_config
from _kernel_consts import _source, kconst

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


def test_a_value_scale_too_small_for_a_rows_factor_is_refused(lib):
    # v_scale over a denominator of up to 2^46 has to be a normal number: one of 1e-38 kept five bits of it
    cfg = msa_config()
    lib.msa_config_default(ctypes.byref(cfg))
    tail = [FAKE, FAKE, FAKE, 4, 9, 100, 1280, 0.088, FAKE, None, FAKE, 0, None]
    for v_scale, code in ((1e-38, SHAPE), (2.0 ** -81, SHAPE), (2.0 ** -80, WORKSPACE), (3e38, WORKSPACE)):
        assert lib.msa_attend_chunk_fp8kv(ctypes.byref(cfg), FAKE, FAKE, FAKE, 1.0, v_scale, *tail) == code, v_scale


def test_the_other_calls_do_without_the_extension_module(monkeypatch):
    # no g++ and no module of this PyTorch and Python: libmsa loads, and only a call that needs the module raises
    monkeypatch.setattr(_build, "GXX", "no-such-compiler")
    monkeypatch.setattr(_build, "ext_path", lambda: os.path.join(_build.BUILD, "no-such-module.so"))
    for name in ("_lib", "_ext"):
        monkeypatch.setattr(binding, name, None)
    assert _build.build() == _build.LIB and _build.up_to_date()
    assert msa.make_config().topk == 16
    x, i = torch.zeros(4, 64, 128, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(RuntimeError, match="no-such-compiler"):
        msa.msa_rotary(x, None, i, torch.zeros(64))
    assert msa.make_config().topk == 16


def test_the_extension_module_is_named_after_python_too():
    name = os.path.basename(_build.ext_path())
    assert torch.__version__ in name and sysconfig.get_config_var("SOABI") in name


def test_libmsa_builds_without_pytorch():
    # (the package itself takes torch tensors; its build does not)
    code = ("import sys, importlib.util as u; sys.modules['torch'] = None; "
            f"s = u.spec_from_file_location('b', {_build.__file__!r}); m = u.module_from_spec(s); s.loader.exec_module(m); "
            "print(m.build())")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == _build.LIB, r.stderr


def test_the_last_blocks_flag_is_read_behind_the_wait_for_its_tile():
    # every lane of the issuing warp reads the flag that the producer wrote before the block's copies: only a lane's own
    # wait for the copies orders its read
    text = _source("chunk_attend.cu")
    a = text.index("const int lv = 2 * base + 2 * nb - 1")
    part = text[a:text.index("fence_proxy_async_smem", a)]
    assert 0 < part.index("ca_wait(&sm.kv_full[sv]") < part.index("keys_of(nb - 1)")


def test_the_rotary_grid_is_resident_at_once(tmp_path):
    # the CTAs per SM that the launch counts on have to fit its 65536 registers and 2048 threads (registers are given to a
    # warp in units of 8 a thread)
    r = subprocess.run([_build._nvcc(), *_build.ARCH, *_build.FLAGS, "-Xptxas", "-v", "-c",
                        os.path.join(_build.CSRC, "rotary.cu"), "-o", str(tmp_path / "rotary.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    regs = max(int(x) for x in re.findall(r"Used (\d+) registers", r.stderr))
    threads = kconst("kRoThreads", "rotary.cu")
    per_sm = re.search(r"per_sm = std::min\((\w+),", _source("rotary.cu")).group(1)
    per_sm = int(per_sm) if per_sm.isdigit() else kconst(per_sm, "rotary.cu")
    assert per_sm * threads <= 2048 and per_sm * threads * (-(-regs // 8) * 8) <= 65536, (per_sm, regs)
