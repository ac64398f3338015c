"""Host check of the GEMM epilogues' output boxes (kd_boxes.h)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_box_is_staged_while_a_transfer_reads_it(tmp_path):
    """Tiles with an odd number of boxes followed by others: the boxes are taken in
    turn over all of a warp's tiles, and a transfer that reads as late as the waits
    allow never finds its box staged again."""
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path / "box_turn_check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror",
                    "-I" + os.path.join(ROOT, "chunked_kl_loss_chunk_b200", "csrc"),
                    os.path.join(ROOT, "tests", "c", "box_turn_check.cc"), "-o", exe],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
