"""What the adapters' host code decides for the kernels, on the CPU under
sanitizers: the layout of a chunk in LDS, and which division of the work a batch
gets."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HC = os.path.join(ROOT, "tests", "host_check")
CSRC = os.path.join(ROOT, "block_quantized_weight_qmat_amd", "csrc")


def run(tmp_path, driver):
    exe = str(tmp_path / "driver")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        f"-I{HC}", f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(HC, driver), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_a_chunk_is_read_inside_its_bytes(tmp_path):
    assert "all reads inside" in run(tmp_path, "lora_layout_driver.cpp")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_the_division_of_batches_of_unlike_sequences(tmp_path):
    assert "all batches as measured" in run(tmp_path, "lora_division_driver.cpp")
