"""The attention kernels' schedule on the host (no GPU): tests/kv_schedule.cu, compiled with the kernels' headers."""
import os
import subprocess

import pytest

from quantized_speculative_decoding_qspec_gb300 import build as b

TESTS = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("kv") / "schedule")
    r = subprocess.run([b.nvcc(), *b.ARCH, "-std=c++17", "-O1", "-I" + b.INCLUDE, "-I" + b.CSRC,
                        os.path.join(TESTS, "kv_schedule.cu"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def test_runs_given_up_leave_no_ticket_behind(program):
    """Runs cover every unit once; when some of them give up, all tickets still return to zero."""
    r = subprocess.run([program], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
    rows = [[int(x) for x in line.split()] for line in r.stdout.splitlines()]
    assert len(rows) >= 30
    assert sum(row[2] > 0 for row in rows) >= 20           # batches with cut items
    assert sum(row[3] > 0 for row in rows) >= 5            # where leaving without the rest would have left tickets
