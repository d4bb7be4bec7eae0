"""The set-up that the decoding libraries share (csrc/host.cuh), compiled
against a fake of the CUDA runtime: failures are made on the host."""
import os
import subprocess

from rotated_w4a4_quantized_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_a_failed_set_up_is_tried_again_and_leaves_no_error(tmp_path):
    exe = str(tmp_path / "host_setup")
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.run(["g++", "-std=c++17", f"-I{cuda}", os.path.join(HERE, "host_setup.cpp"), "-o", exe], check=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.stdout.strip() == "ok" and run.returncode == 0, run.stdout
