"""The dense operators' register loads on the host: the kernels' own code
(dense_load.h) over matrices between unmapped pages, at every small pitch and
every remainder of the summed length."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_loads_stay_inside_the_matrix(tmp_path):
    exe = str(tmp_path / "dense_load_check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-w", "-I", os.path.join(ROOT, "unet_x3_convolution_amd", "csrc"),
                    os.path.join(ROOT, "tests", "dense_load_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
