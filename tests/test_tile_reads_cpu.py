"""CPU-only: no transfer of a tile reads outside its operand. tile_reads.cpp runs the loaders of
csrc/mm_tile.h on the host, lane by lane."""
import os
import subprocess

from tensor_gradient_compression_amd import build


def test_tiles_read_inside_their_operands(tmp_path):
    src, exe = os.path.join(os.path.dirname(os.path.abspath(__file__)), "tile_reads.cpp"), str(tmp_path / "tile_reads")
    made = subprocess.run([build._hipcc(), "-x", "hip", "--offload-host-only", "-O2", "-std=c++17", "-I", build.INCLUDE,
                           "-I", build.CSRC, src, "-o", exe], capture_output=True, text=True)
    assert made.returncode == 0, made.stdout + made.stderr
    ran = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert ran.returncode == 0, ran.stdout
