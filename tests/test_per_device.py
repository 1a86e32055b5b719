"""Kernel attributes are set once per device, not once per process: the bookkeeping
(csrc/mxq_per_device.h), and that no launch keeps a result of its own for all devices."""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp8_activation_quant_gb300", "csrc")


def test_once_per_device(tmp_path):
    exe = str(tmp_path / "per_device_check")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", CSRC, os.path.join(os.path.dirname(__file__), "per_device_check.cpp"),
                    "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_attributes_are_not_kept_for_the_process():
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        assert not re.search(r"static\s+(const\s+)?cudaError_t\s+\w+\s*=", text), name
        # every limit is set through the helper
        assert text.count("cudaFuncSetAttribute(") == (1 if name == "mxq_internal.h" else 0), name
