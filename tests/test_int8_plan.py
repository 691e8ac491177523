"""The int8 products' plans, walked on the CPU (tests/int8_plan_sweep.cpp)."""

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_unit_has_one_owner_and_every_piece_its_place(tmp_path):
    exe = str(tmp_path / "sweep")
    csrc = os.path.join(HERE, "..", "nvfp4_weight_dense_amd", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", csrc, os.path.join(HERE, "int8_plan_sweep.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok "), r.stdout + r.stderr
