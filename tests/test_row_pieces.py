"""The row kernels' address arithmetic on the host: no window reads past the
last row that has to exist, and every column is taken once."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_windows_stay_in_the_rows_that_exist(tmp_path):
    exe = str(tmp_path / "pieces_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "zero_sharded_optimizer_flatten_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "c", "pieces_check.cpp"), "-o", exe], check=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout
    assert int(run.stdout) > 100_000
