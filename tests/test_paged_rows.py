"""From a row of the packed queries to its token, for starts that cannot be
(csrc/paged_index.h), compiled for the host with overflows trapped."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_rows_lead_to_tokens_or_nowhere(tmp_path):
    exe = str(tmp_path / "paged_rows_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror",
                    "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    os.path.join(HERE, "paged_rows_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_the_write_takes_the_checked_step():
    """The kernel forms no token number of its own."""
    with open(os.path.join(HERE, "..", "dual_window_attention_b200", "csrc", "paged_append.cuh")) as f:
        source = f.read()
    assert "row_token(sp, row)" in source and "row - sp.q0" not in source
