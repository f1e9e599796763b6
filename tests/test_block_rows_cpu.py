"""The norms' rows on the CPU, for every row length: copies inside their tensors and places, groups
inside their copies, every column in one thread's hands, two places for every block that has more
than one row, shared memory within an SM's."""

import os
import subprocess

from recurrent_associative_memory_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_addresses_of_every_row_length(tmp_path):
    program = str(tmp_path / "check")
    subprocess.run([build.nvcc(), *build.ARCH, "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-I", build.CSRC,
                    os.path.join(HERE, "block_norm_rows_check.cu"), "-o", program], check=True, capture_output=True, text=True)
    r = subprocess.run([program], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout, r.stderr)
