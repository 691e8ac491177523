"""Every kernel that an int8 product's plan can choose is run by a GPU test: the sizes of tests/int8_shapes.py reach
each class that a sweep of sizes meets (tests/int8_plan_classes.cpp)."""

import os
import subprocess

import int8_shapes as shapes

HERE = os.path.dirname(os.path.abspath(__file__))


def test_the_sizes_reach_every_kernel(tmp_path):
    exe = str(tmp_path / "classes")
    csrc = os.path.join(HERE, "..", "nvfp4_weight_dense_amd", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", csrc, os.path.join(HERE, "int8_plan_classes.cpp"), "-o", exe], check=True)
    sizes = "".join("%d %d %d %d\n" % (*s, x) for x, of in ((1, shapes.ONE), (2, shapes.TWO)) for s in of)
    run = set(subprocess.run([exe, "of"], input=sizes, capture_output=True, text=True, check=True).stdout.split())
    met = [line.split() for line in subprocess.run([exe, "all"], capture_output=True, text=True, check=True).stdout.splitlines()]
    assert len(met) > 50
    missing = [" ".join(c) for c in met if c[0] not in run]
    assert not missing, "no size runs (class, and a size that does):\n" + "\n".join(missing)
