"""The index arithmetic of the paged attention (csrc/paged_index.h), compiled for
the host and checked exhaustively on small ranges."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_index_arithmetic(tmp_path):
    exe = str(tmp_path / "paged_index_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    os.path.join(HERE, "paged_index_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_unit_slots(tmp_path):
    exe = str(tmp_path / "paged_units_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    os.path.join(HERE, "paged_units_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
