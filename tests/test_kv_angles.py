"""The frequency table at far positions, against angles worked out with 60 decimals (no GPU)."""
from decimal import Decimal, getcontext

import numpy as np
import pytest

from quantized_speculative_decoding_qspec_gb300 import qspec as q


@pytest.fixture(scope="module", autouse=True)
def lib():
    import __graft_entry__ as g
    g.build()
    return q.load()


def pi():
    """Machin's formula."""
    def arctan_inv(n):
        x = Decimal(1) / n
        total, term, k = x, x, 1
        while abs(term) > Decimal(10) ** -70:
            term /= -n * n
            k += 2
            total += term / k
        return total
    return 4 * (4 * arctan_inv(5) - arctan_inv(239))


@pytest.mark.parametrize("base,rot", [(10000, 128), (500000, 64)])
def test_far_angles(base, rot):
    """position * word / 2^64 turns against position * base^(-2i/rot) / (2 pi): a word is off by its own last bit and a
    few fp64 roundings (16 of them) of a frequency below a sixth of a turn, which the position multiplies."""
    getcontext().prec = 80
    two_pi = 2 * pi()
    words = q.qspec_rotary_turns(rot, float(base))[0].numpy().view(np.uint64)
    for i in range(rot // 2):
        w = (Decimal(base).ln() * (-2 * i) / rot).exp() / two_pi
        for pos in (1, 8191, 10 ** 6 + 1, 2 ** 31 - 1, -5):
            got = Decimal((pos * int(words[i])) % 2 ** 64) / 2 ** 64
            off = (got - (pos * w) % 1) % 1
            off = min(off, 1 - off)
            assert off <= abs(pos) * (w * 16 / 2 ** 53 + Decimal(2) ** -64), (i, pos, off)
