"""What a pair of CTAs waits for after a wait that gave up, on the host: every
ending of its copies, with the barriers played."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_nothing_stays_in_flight_and_every_wait_ends(tmp_path):
    exe = str(tmp_path / "drain_check")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "zero_sharded_optimizer_flatten_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "c", "drain_check.cpp"), "-o", exe], check=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout
    assert int(run.stdout) > 10_000
