"""How the root-mean-square norm deals rows out to threads (host arithmetic),
over all widths and the row counts where it changes, and its backward pass
without rows."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "scaled_fp8_gemm_amd", "csrc")


def test_row_shapes_of_all_widths(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    exe = str(tmp_path / "rms_shape_check")
    subprocess.check_call([gxx, "-O1", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC,
                           os.path.join(HERE, "rms_shape_check.cpp"), "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stdout)


@pytest.mark.parametrize("cols", [40, 8192, 8193, 12288, 16385, 32768])
def test_backward_without_rows_reaches_the_launch(cols):
    """rows = 0 needs no device memory but the sums'; where there is no device
    the launch is refused (FP8_ERR_HIP = 5).  In a process of its own, which an
    arithmetic fault would end."""
    if torch.cuda.is_available():
        pytest.skip("its pointers are not device memory")
    code = ("from scaled_fp8_gemm_amd import fp8sg as F\n"
            "p = 0x10000\n"
            "print(F.lib().fp8_rmsnorm_bwd(None, None, 0, None, None, p, 0, None, 0, %d, None, p,"
            " p, None))" % cols)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(HERE))
    assert r.returncode == 0 and r.stdout.split() == ["5"], (r.returncode, r.stdout, r.stderr)
