"""What include/attn.h promises and the host can show: the oracle's readings of it, and refusals."""
import numpy as np

from oracle import attn as A


def test_oracle_ranks_protected_slots_by_weight():
    acc, pos = [9.0, 1.0, 5.0, 7.0, 3.0], [0, 1, 2, 3, 4]
    assert A.evict(acc, pos, 3, 0, 5, 5)[0].tolist() == [0, 3, 2]
    # two of three protected slots stay: NaN last, and no other slot whatever its weight
    assert A.evict([np.nan, 0.0, 100.0, -1.0], [0, 1, 2, 3], 2, 2, 1, 4)[0].tolist() == [3, 1]
    assert A.evict([np.nan, np.nan, 100.0, -1.0], [0, 1, 2, 3], 2, 2, 1, 4)[0].tolist() == [0, 3]
