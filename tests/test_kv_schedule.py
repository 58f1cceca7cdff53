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
    rows = [[int(x) for x in line.split()] for line in r.stdout.splitlines() if not line.startswith("ctas")]
    assert len(rows) >= 30
    assert sum(row[2] > 0 for row in rows) >= 20           # batches with cut items
    assert sum(row[3] > 0 for row in rows) >= 5            # where leaving without the rest would have left tickets


def test_every_cta_of_a_decode_grid_is_resident(program):
    """228 KB of shared memory an SM, 1 KB of it taken by each CTA: the CTAs that share the work out must all fit, and
    one more must not where the grid is smaller than the four (or two) that registers allow."""
    r = subprocess.run([program], capture_output=True, text=True, timeout=60)
    rows = [[int(x) for x in line.split()[1:]] for line in r.stdout.splitlines() if line.startswith("ctas")]
    assert len(rows) == 32
    for D, RG, B, ctas, smem in rows:
        each = -(-smem // 128) * 128 + 1024
        assert 1 <= ctas <= 4 // RG and ctas * each <= 228 * 1024, (D, RG, B, ctas, smem)
        assert ctas == 4 // RG or (ctas + 1) * each > 228 * 1024, (D, RG, B, ctas, smem)
