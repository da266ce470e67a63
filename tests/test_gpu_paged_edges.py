"""The paged decode where it can go wrong: slots and queries that are reused
row after row, copies in flight when a wait expires, V rows of very different
magnitudes, infinities.  Against the oracle, as tests/test_gpu_paged.py."""
import numpy as np
import pytest

from paged_helpers import Paged
from test_gpu_paged import FORMATS, _decode

pytestmark = pytest.mark.gpu


@FORMATS
@pytest.mark.parametrize("nq,hd", [(8, 128), (16, 256)])
def test_slots_and_queries_reused_by_row_after_row(nq, hd, e4m3):
    """More rows than warps, nearly all of which end inside a tile: each warp
    clears the tail of a V slot, refills the slot and (16 heads of 256) takes
    the next row's Q into shared memory, again and again.  The same bits every
    time, within the bound."""
    rng = np.random.default_rng(31)
    lens = [int(n) for n in rng.integers(1, 150, 1400)]
    c = Paged(1, hd, 16, lens, e4m3, seed=31)
    c.fill(rng, lens)
    c.upload()
    first = _decode(c, nq, lens)
    for _ in range(5):
        again = _decode(c, nq, lens)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])
