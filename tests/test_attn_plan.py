"""How attention's work is divided, on the CPU: a sanitizer build of the plan over
the arguments that qmat_attn accepts, from one token to the limits."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HC = os.path.join(ROOT, "tests", "host_check")
CSRC = os.path.join(ROOT, "block_quantized_weight_qmat_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_plan_under_sanitizers(tmp_path):
    exe = str(tmp_path / "attn_plan_drv")
    r = subprocess.run(["g++", "-std=c++17", "-O0", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(HC, "attn_plan_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all plans ok" in r.stdout, r.stdout + r.stderr
