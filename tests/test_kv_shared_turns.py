"""The order of a shared item's key tiles on the host (no GPU): tests/kv_shared_turns.cu, compiled with the kernels' headers."""
import os
import subprocess

from quantized_speculative_decoding_qspec_gb300 import build as b

TESTS = os.path.dirname(os.path.abspath(__file__))


def test_every_tile_is_taken_once_and_none_of_an_item_that_sees_nothing(tmp_path):
    exe = str(tmp_path / "turns")
    r = subprocess.run([b.nvcc(), *b.ARCH, "-std=c++17", "-O1", "-I" + b.INCLUDE, "-I" + b.CSRC,
                        os.path.join(TESTS, "kv_shared_turns.cu"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "ok\n", (r.returncode, r.stdout)
