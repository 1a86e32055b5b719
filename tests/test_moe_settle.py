"""The experts' GEMMs after a wait that ran out: what the loads in flight still owe a stage's barrier
(csrc/mxq_settle.h), over random points at which the loaders stop. Host arithmetic only."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_copy_in_flight_is_waited_for(tmp_path):
    exe = str(tmp_path / "settle_sim")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "mxfp8_activation_quant_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "settle_sim.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout) > 1000  # stages whose barrier, left alone, would not have completed
