"""The KV-cache entry points on the CPU: refused arguments (through the built
library, and through a sanitizer build of the C ABI with stub launchers), the
workspace size, and the binding's own checks."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from block_quantized_weight_qmat_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HC = os.path.join(ROOT, "tests", "host_check")
CSRC = os.path.join(ROOT, "block_quantized_weight_qmat_amd", "csrc")
OK, E_FMT, E_SHAPE, E_NULL, E_ALIGN, E_WORKSPACE, E_DTYPE = 0, 1, 2, 3, 5, 7, 8
A = 0x10000  # a 16-byte aligned fake address: never dereferenced (rejected first)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.library_path()):
        pytest.skip("libqmat.so not built")
    return binding.load_library()


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_kv_abi_checks_under_sanitizers(tmp_path):
    exe = str(tmp_path / "kv_abi_drv")
    r = subprocess.run(
        ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
         f"-I{HC}", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", "-x", "c++", os.path.join(CSRC, "qmat_api.cpp"),
         os.path.join(CSRC, "qmat_kv_api.cpp"), os.path.join(HC, "launch_stub.cpp"),
         os.path.join(HC, "kv_launch_stub.cpp"), os.path.join(HC, "kv_abi_driver.cpp"), "-o", exe],
        capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all cases ok" in r.stdout, r.stdout + r.stderr


def args(**kw):
    a = binding.AttnArgs()
    base = dict(k_fmt=0, v_fmt=1, dtype=0, causal=1, q=A, out=A, k_cache=A, v_cache=A, page_table=A, q_start=A, kv_len=A,
                q_stride=1024, out_stride=1024, n_tokens=4, n_seqs=4, max_q=1, max_kv=100, heads=8, kv_heads=2,
                head_dim=128, cells=4096, page_size=16, pages_per_seq=4096, window=0, scale=0.1)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


def test_struct_and_strings(lib):
    assert ctypes.sizeof(binding.AttnArgs) == 4 * 4 + 7 * 8 + 13 * 8 + 8
    assert lib.qmat_strerror(E_DTYPE) != b"unknown status"
    assert b"element type" in lib.qmat_strerror(E_DTYPE)


def test_attn_refusals(lib):
    def call(**kw):
        return lib.qmat_attn(ctypes.byref(args(**kw)), None, 0, None)
    assert call(k_fmt=2) == E_FMT and call(v_fmt=-1) == E_FMT and call(dtype=7) == E_DTYPE
    for kw in (dict(head_dim=32), dict(head_dim=96), dict(heads=9), dict(kv_heads=0), dict(page_size=48),
               dict(page_size=0), dict(window=-1), dict(q_stride=8), dict(scale=float("nan")), dict(max_q=-1),
               dict(pages_per_seq=2 ** 27), dict(cells=2 ** 31), dict(n_tokens=2 ** 25)):
        assert call(**kw) == E_SHAPE, kw
        assert lib.qmat_attn_workspace_bytes(ctypes.byref(args(**kw))) == -1, kw
    assert call(q=None) == E_NULL and call(kv_len=None) == E_NULL and call(k_cache=None) == E_NULL
    assert call(out=A + 4) == E_ALIGN and call(out_stride=1026) == E_ALIGN
    assert call(n_tokens=0, q=None) == OK and call(n_seqs=0) == OK
    assert lib.qmat_attn(None, None, 0, None) == E_NULL


def test_attn_workspace(lib):
    """0 where nothing is split; whole partial rows where a sequence is; refused when too small."""
    def need(**kw):
        return lib.qmat_attn_workspace_bytes(ctypes.byref(args(**kw)))
    assert need() == 0 and need(max_kv=0) == 0
    n = need(n_seqs=1, n_tokens=1, max_kv=60000)
    assert n > 0 and n % 4 == 0
    assert need(n_seqs=1, n_tokens=1, max_kv=2 ** 62) == need(n_seqs=1, n_tokens=1, max_kv=65536)  # the table's cells
    assert need(n_seqs=1, n_tokens=1, max_kv=60000, window=64) == 0  # few cells to see
    a = args(n_seqs=1, n_tokens=1, max_kv=60000)
    assert lib.qmat_attn(ctypes.byref(a), None, n, None) == E_WORKSPACE
    assert lib.qmat_attn(ctypes.byref(a), A, n - 1, None) == E_WORKSPACE
    assert lib.qmat_attn(ctypes.byref(a), A + 4, n, None) == E_ALIGN
    # every shape that the checks let through has a size that fits
    for kw in (dict(n_seqs=2 ** 24, n_tokens=2 ** 24, max_q=2 ** 24, heads=32, kv_heads=1, q_stride=4096, out_stride=4096),
               dict(heads=4096, kv_heads=4096, q_stride=2 ** 19, out_stride=2 ** 19, max_kv=2 ** 40, page_size=2 ** 18)):
        assert need(**kw) >= 0, kw


def test_binding_refuses_cpu_tensors_and_types():
    t = torch.zeros
    with pytest.raises(TypeError):
        binding.kv_store("q4_0", "q4_0", t(2, 64), t(2, 64), t(2, dtype=torch.int32), t(4, 36, dtype=torch.uint8),
                         t(4, 36, dtype=torch.uint8))
    with pytest.raises(TypeError):
        binding.kv_load("q4_0", "q4_0", t(4, 36, dtype=torch.uint8), t(4, 36, dtype=torch.uint8),
                        t(2, dtype=torch.int32), 64)
    with pytest.raises(TypeError):
        binding.attn("q4_0", "q4_0", t(1, 2, 64), t(16, 36, dtype=torch.uint8), t(16, 36, dtype=torch.uint8),
                     t(1, 1, dtype=torch.int32), t(2, dtype=torch.int32), t(1, dtype=torch.int32), 1, 16)
    with pytest.raises(TypeError):
        binding.attn("q4_0", "q4_0", t(1, 2, 64, dtype=torch.float64), t(16, 36, dtype=torch.uint8),
                     t(16, 36, dtype=torch.uint8), t(1, 1, dtype=torch.int32), t(2, dtype=torch.int32),
                     t(1, dtype=torch.int32), 1, 16)
