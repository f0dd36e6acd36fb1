"""The RMS norm kernels' row index arithmetic (gb_rows.cuh) on the CPU: no thread of any small shape's teams reads
a vector beyond the tensor, and every element of a row is one thread's."""
import os
import subprocess

from cross_vendor_gradient_gb300 import build as gbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_read_of_a_row_lies_within_the_tensor(tmp_path):
    exe = str(tmp_path / "rows_host")
    subprocess.run([gbuild.nvcc(), *gbuild.ARCH, "-O2", "-std=c++17", "-I", gbuild.CSRC, "-o", exe,
                    os.path.join(ROOT, "tests", "rows_host.cu")], check=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout
    assert int(run.stdout.split()[1]) > 10_000


def test_rows_before_the_last_that_the_end_of_the_tensor_cuts():
    """By the definition alone: a row is cut when the vector of 8 that holds its last element ends beyond the tensor.
    Widths of 1, 2, 3 and 5 have such rows before the last one."""
    widths = set()
    for cols in range(1, 64):
        for rows in range(1, 70):
            n = rows * cols
            for row in range(rows):
                ends = ((row + 1) * cols + 7) // 8 * 8
                assert (ends > n) == (row >= n // 8 * 8 // cols)
                if ends > n and row + 1 < rows:
                    widths.add(cols)
    assert widths == {1, 2, 3, 5}
