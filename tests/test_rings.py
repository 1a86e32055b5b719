"""The attention's rings (csrc/mxq_rings.h): no wait by parity passes a phase too early, in whatever order loads land and the
two sets of warps get on. Host arithmetic only."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_wait_passes_early(tmp_path):
    exe = str(tmp_path / "ring_sim")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-I", os.path.join(ROOT, "mxfp8_activation_quant_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "ring_sim.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert all(int(n) > 0 for n in r.stdout.split())  # rings outside the rule do pass early
