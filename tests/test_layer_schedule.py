"""Index arithmetic of the layer's kernels replayed on the host, compiled from their own headers. No kernel runs."""
import os
import subprocess

from compressed_sgd_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def replay(name, tmp_path):
    exe = str(tmp_path / name)
    subprocess.check_call([build.nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC,
                           "-o", exe, os.path.join(HERE, name + ".cu")])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    return r.stdout


def test_every_block_is_taken_once_and_joined(tmp_path):
    """The schedule of the products' tiles, with every number of stacked tiles and some thousand others."""
    assert int(replay("tiles_replay", tmp_path).split()[0]) > 9000


def test_whole_groups_of_a_row_lie_in_it(tmp_path):
    """The norm's weight between boundaries."""
    replay("entries_replay", tmp_path)
