"""The division of the key-weight kernel's work, on the host: the header that the kernel
uses, compiled as plain C++ (no GPU)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_part_of_a_tile_has_a_row_block(tmp_path):
    """The kernel's barrier between two requests of a CTA pair relies on it; the rings of
    every row count fit in shared memory."""
    exe = str(tmp_path / "kw_plan")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-x", "c++",
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "speculative_decoding_tree_va_b200", "csrc"),
                    os.path.join(ROOT, "tests", "c", "kw_plan.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
