"""HistoryStore.commit refuses rows and states of another type or shape before it reserves anything (on the
CPU: nothing reaches the library)."""
import pytest
import torch

from tree_forked_decision_b200 import inputs
from tree_forked_decision_b200.history import HistoryStore


def _rows(n=5, h=2, d=8, dtype=torch.bfloat16):
    return torch.zeros(n, h, d, dtype=dtype)


@pytest.mark.parametrize("k,v,state,error", [
    (_rows(dtype=torch.float32), _rows(dtype=torch.float32), None, TypeError),
    (_rows(), _rows(dtype=torch.float32), None, TypeError),
    (_rows(h=3), _rows(h=3), None, TypeError),
    (_rows(d=16), _rows(), None, TypeError),
    (_rows(4), _rows(4), None, ValueError),
    (_rows(), _rows(4), None, ValueError),
    (_rows(), _rows(), torch.zeros(2, 1, 32, 16), TypeError),
    (_rows(), _rows(), torch.zeros(2, 1, 32, 32, dtype=torch.float64), TypeError),
])
def test_commit_refuses(k, v, state, error):
    store = HistoryStore(n_blocks=4, block_rows=16, max_requests=2, max_blocks=3, Hkv=2, d=8, H=1, dk=32, dv=32,
                         device="cpu")
    with pytest.raises(error):
        store.commit([1], inputs._tree([(0, [(-1, 5)])], 0), None, k, v, state)
    assert store.length(1) == 0 and store.free_blocks() == 4
