"""The schedule of attention over shared prefixes on the host (no GPU): tests/kv_shared_schedule.cu, compiled with the kernels' headers."""
import os
import subprocess

from quantized_speculative_decoding_qspec_gb300 import build as b

TESTS = os.path.dirname(os.path.abspath(__file__))


def test_runs_cover_every_tile_once_and_tiles_what_rows_see(tmp_path):
    exe = str(tmp_path / "schedule")
    r = subprocess.run([b.nvcc(), *b.ARCH, "-std=c++17", "-O1", "-I" + b.INCLUDE, "-I" + b.CSRC,
                        os.path.join(TESTS, "kv_shared_schedule.cu"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
    rows = [[int(x) for x in line.split()] for line in r.stdout.splitlines()]
    assert len(rows) >= 120 and sum(row[2] > 0 for row in rows) >= 80
