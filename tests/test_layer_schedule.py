"""The schedule of the products' tiles, replayed on the host with every number of tiles: compiled from the kernels' own header. No
kernel runs."""
import os
import subprocess

from compressed_sgd_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_block_is_taken_once_and_joined(tmp_path):
    exe = str(tmp_path / "tiles_replay")
    subprocess.check_call([build.nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC,
                           "-o", exe, os.path.join(HERE, "tiles_replay.cu")])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout.split()[0]) > 9000
