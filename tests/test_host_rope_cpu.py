"""The norm and rotation's arguments as the kernel gets them, and its split of
a token's heads, compiled and run on the CPU (``tests/host/rope_args_check.cu``).  Needs nvcc only."""
import os
import shutil
import subprocess
import tempfile

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
NVCC = next((c for c in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc") if c and os.path.exists(c)), None)


@pytest.mark.skipif(NVCC is None, reason="nvcc not available")
def test_a_side_without_heads_leaves_nothing_in_the_arguments():
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "rope_args_check")
        subprocess.run([NVCC, "-std=c++17", "-O1",
                        "-I", os.path.join(ROOT, "compressed_decode_attention_encode_b200", "csrc"),
                        os.path.join(HERE, "host", "rope_args_check.cu"), "-o", exe], check=True, capture_output=True)
        out = subprocess.run([exe], capture_output=True, text=True)
        assert out.returncode == 0, out.stdout + out.stderr
