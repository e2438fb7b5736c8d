"""Windows with sinks on the CPU: what the kernels compute of their work units, compiled for the host."""

import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def walk(name, tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    exe = str(tmp_path / name)
    run = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O1", "-std=c++17",
                          "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include"),
                          "-I" + os.path.join(ROOT, "attention_sm_flashattention_gb300", "csrc"),
                          os.path.join(ROOT, "tests", name + ".cu"), "-o", exe], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout


def test_steps_of_the_dq_kernels(tmp_path):
    walk("sink_steps", tmp_path)


def test_far_units_in_closed_form(tmp_path):
    walk("sink_far", tmp_path)
