"""What include/attn.h promises and the host can show: the oracle's readings of it, and refusals."""
import types

import numpy as np
import pytest

from block_scaled_fp4_softmax_gb300 import attn
from oracle import attn as A


def test_oracle_ranks_protected_slots_by_weight():
    acc, pos = [9.0, 1.0, 5.0, 7.0, 3.0], [0, 1, 2, 3, 4]
    assert A.evict(acc, pos, 3, 0, 5, 5)[0].tolist() == [0, 3, 2]
    # two of three protected slots stay: NaN last, and no other slot whatever its weight
    assert A.evict([np.nan, 0.0, 100.0, -1.0], [0, 1, 2, 3], 2, 2, 1, 4)[0].tolist() == [3, 1]
    assert A.evict([np.nan, np.nan, 100.0, -1.0], [0, 1, 2, 3], 2, 2, 1, 4)[0].tolist() == [0, 3]


CALLS = {
    "rope": lambda c, **kw: attn.attn_qk_norm_rope(None, None, None, None, None, None, c, None, **kw),
    "tree": lambda c, **kw: attn.attn_tree_decode(None, None, None, c, **kw),
    "weights": lambda c, **kw: attn.attn_cache_weights(None, None, None, None, c, None, **kw),
    "evict": lambda c, **kw: attn.attn_cache_evict(c, None, None, None, None, 8, **kw),
}


@pytest.mark.parametrize("call", CALLS)
def test_a_cache_of_another_device_is_refused(call, monkeypatch):
    """Nothing is looked at, allocated or launched before."""
    cache = types.SimpleNamespace(index=1, device="cuda:1")
    monkeypatch.setattr(attn, "_current", lambda: 0)
    with pytest.raises(attn.MoeError, match="cuda:0 is current"):
        CALLS[call](cache)
    monkeypatch.setattr(attn, "_current", lambda: 1)
    with pytest.raises(attn.MoeError, match="the stream on cuda:0"):
        CALLS[call](cache, stream=types.SimpleNamespace(device_index=0, cuda_stream=7))
