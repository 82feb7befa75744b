"""The general ragged kernel's operand loads, run on the host: no thread reads
outside a matrix, at any width, tile and number of rows around a stage (no GPU
needed)."""
import os
import subprocess

from round_dropless_expert_amd.csrc import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_operand_loads_stay_inside_their_matrices(tmp_path):
    exe = str(tmp_path / "operand_bounds")
    subprocess.run([build.HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O2", "-Wall",
                    os.path.join(HERE, "operand_bounds.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
