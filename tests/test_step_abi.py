"""The entry points of a step on the CPU: refused arguments (through a
sanitizer build of the C ABI with stub launchers), and the binding's own
checks."""
import os
import shutil
import subprocess

import pytest
import torch

from block_quantized_weight_qmat_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HC = os.path.join(ROOT, "tests", "host_check")
CSRC = os.path.join(ROOT, "block_quantized_weight_qmat_amd", "csrc")

needs_lib = pytest.mark.skipif(not os.path.exists(binding.library_path()), reason="libqmat.so not built")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_step_abi_checks_under_sanitizers(tmp_path):
    exe = str(tmp_path / "step_abi_drv")
    r = subprocess.run(
        ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
         f"-I{HC}", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", "-x", "c++", os.path.join(CSRC, "qmat_api.cpp"),
         os.path.join(CSRC, "qmat_step_api.cpp"), os.path.join(HC, "launch_stub.cpp"),
         os.path.join(HC, "step_launch_stub.cpp"), os.path.join(HC, "step_abi_driver.cpp"), "-o", exe],
        capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all cases ok" in r.stdout, r.stdout + r.stderr


@needs_lib
def test_embed_refuses_cpu_tensors_and_types():
    t = torch.zeros(4, 34, dtype=torch.uint8)
    with pytest.raises(TypeError):
        binding.embed("q8_0", t, 32)
    with pytest.raises(TypeError):
        binding.embed("q8_0", t.float(), 32)
    with pytest.raises(KeyError):
        binding.embed("q5_0", t, 32)


@needs_lib
def test_rms_norm_refuses():
    x, w = torch.zeros(2, 64), torch.ones(64)
    with pytest.raises(TypeError):
        binding.rms_norm(x, w)
    with pytest.raises(TypeError):
        binding.rms_norm(x.double(), w)
    with pytest.raises(ValueError):
        binding.rms_norm(x, w, want="none")
    with pytest.raises(ValueError):
        binding.rms_norm(x[0], w)


def test_rope_tables():
    """The frequencies in 64 bits, and pairs shared out over axes one after the other or in turn."""
    f = binding.rope_freq(8, base=10000.0, device="cpu")
    assert f.dtype == torch.float64 and f.tolist() == [1.0, 10000.0 ** -0.25, 10000.0 ** -0.5, 10000.0 ** -0.75]
    assert binding.rope_axis([1, 2, 3], device="cpu").tolist() == [0, 1, 1, 2, 2, 2]
    assert binding.rope_axis([3, 2, 1], cycle=True, device="cpu").tolist() == [0, 1, 2, 0, 1, 0]
    assert binding.rope_axis([], device="cpu").numel() == 0
    with pytest.raises(ValueError):
        binding.rope_freq(7, device="cpu")
    with pytest.raises(ValueError):
        binding.rope_axis([2, -1], device="cpu")


@needs_lib
def test_rope_refuses():
    q, pos, freq = torch.zeros(3, 2, 16), torch.zeros(3, dtype=torch.int32), torch.ones(8, dtype=torch.float64)
    with pytest.raises(TypeError):
        binding.rope(q, None, pos, freq)
    with pytest.raises(TypeError):
        binding.rope(q.double(), None, pos, freq)
    with pytest.raises(ValueError):
        binding.rope(q[0], None, pos, freq)


@needs_lib
def test_page_step_refuses():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        binding.page_step(i, i, i.view(2, 1), i, i[:1], 16, 4)
    with pytest.raises(TypeError):
        binding.page_step(i.long(), i, i.view(2, 1), i, i[:1], 16, 4)


def test_structs_have_the_headers_sizes():
    """Fields of 8 bytes follow each other without gaps; the 32-bit ones come first."""
    import ctypes
    assert ctypes.sizeof(binding.NormArgs) == 8 + 6 * 8 + 6 * 8 + 8
    assert ctypes.sizeof(binding.RopeArgs) == 4 * 4 + 9 * 8 + 10 * 8 + 8
    assert ctypes.sizeof(binding.PageArgs) == 11 * 8 + 5 * 8
    assert ctypes.sizeof(binding.LoraArgs) == 8 + 9 * 8 + 9 * 8


@needs_lib
def test_lora_refuses():
    t = torch.zeros
    i = t(2, dtype=torch.int32)
    args = (t(2, 34, dtype=torch.uint8), t(1, 8, 32).half(), t(1, 4, 8).half(), i, t(3, dtype=torch.int32), t(2, 4))
    with pytest.raises(TypeError):
        binding.lora(*args)
    with pytest.raises(TypeError):
        binding.lora(args[0], args[1].float(), *args[2:])
