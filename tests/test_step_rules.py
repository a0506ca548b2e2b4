"""A step's calls whose arguments are each allowed and together are not: refused
on the CPU, through a sanitizer build of the C ABI with stub launchers."""
import os
import shutil
import subprocess

import pytest

from block_quantized_weight_qmat_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HC = os.path.join(ROOT, "tests", "host_check")
CSRC = os.path.join(ROOT, "block_quantized_weight_qmat_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_refused_together(tmp_path):
    exe = str(tmp_path / "step_rules")
    r = subprocess.run(
        ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
         f"-I{HC}", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", "-x", "c++", os.path.join(CSRC, "qmat_api.cpp"),
         os.path.join(CSRC, "qmat_step_api.cpp"), os.path.join(HC, "launch_stub.cpp"),
         os.path.join(HC, "step_launch_stub.cpp"), os.path.join(HC, "step_rules_driver.cpp"), "-o", exe],
        capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all cases ok" in r.stdout, r.stdout + r.stderr


@pytest.mark.skipif(not os.path.exists(binding.library_path()), reason="libqmat.so not built")
def test_alignment_is_named_as_the_calls_ask_it():
    """Lists of integers need 4 bytes in some calls, row strides 16: the status' text does not say 16 bytes for all."""
    text = binding.load_library().qmat_strerror(5).decode()
    assert "16" in text and "4" in text and "stride" in text
