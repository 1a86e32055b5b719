"""The attention's roles after a wait that ran out: every one of them ends, and no load is announced over one in flight, wherever the
wait was. Host arithmetic only."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_role_ends(tmp_path):
    exe = str(tmp_path / "giveup_sim")
    subprocess.run(["g++", "-std=c++20", "-O1", "-Wall", "-I", os.path.join(ROOT, "mxfp8_activation_quant_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "giveup_sim.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert all(int(n) > 0 for n in r.stdout.split())  # without the rules some do not
