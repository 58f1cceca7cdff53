"""A beam workspace serves every shape that is no larger in any of its numbers (no GPU: sizes alone)."""
import pytest

from quantized_speculative_decoding_qspec_gb300 import qspec as q


@pytest.fixture(scope="module")
def size():
    import __graft_entry__ as g
    g.build()
    return q.load().qspec_beam_workspace_size


BATCHES = (1, 2, 3, 5, 7, 10, 18, 19, 37, 38, 64, 75, 77, 100, 148, 151, 152, 153, 320)
BEAMS = (1, 2, 3, 4, 5, 8, 9, 17, 32)


@pytest.mark.parametrize("V,n", [(4097, 1), (32000, 64), (128256, 8), (1 << 24, 64)])
def test_smaller_batches_and_fewer_beams_need_no_more(size, V, n):
    table = [[size(B, K, V, n) for B in BATCHES] for K in BEAMS]
    for K, row, fewer in zip(BEAMS, table, [[1] * len(BATCHES)] + table):
        assert row == sorted(row), K
        assert all(a <= b for a, b in zip(fewer, row)), K


@pytest.mark.parametrize("B,K", [(1, 1), (7, 5), (37, 4), (64, 8), (151, 1), (65535, 1)])
def test_smaller_vocabularies_and_fewer_candidates_need_no_more(size, B, K):
    by_V = [size(B, K, V, 64) for V in (64, 4095, 4096, 4097, 8192, 8193, 12289, 32000, 50001, 128256, 152064, 1 << 20, 1 << 24)]
    assert 0 < by_V[0] and by_V == sorted(by_V)
    by_n = [size(B, K, 32000, n) for n in (1, 2, 3, 31, 32, 33, 64)]
    assert by_n == sorted(by_n)


@pytest.mark.parametrize("K,V", [(4, 128256), (1, 128256), (5, 32000)])
def test_a_server_that_allocates_for_its_largest_batch(size, K, V):
    most = size(64, K, V, 8)
    assert all(size(B, K, V, 8) <= most for B in range(1, 65))
