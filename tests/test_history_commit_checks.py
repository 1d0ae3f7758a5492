"""HistoryStore.commit refuses rows and states of another type or shape before it reserves anything (on the
CPU: nothing reaches the library)."""
import pytest
import torch

from tree_forked_decision_b200 import flide, inputs
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


def _fresh():
    store = HistoryStore(n_blocks=4, block_rows=16, max_requests=2, max_blocks=3, Hkv=2, d=8, device="cpu")
    store.mass = torch.arange(96.0).view(2, 48)
    store._weighed = {1: torch.full((0,), 7.0)}  # as accumulate_mass leaves it for an empty slot
    return store


@pytest.mark.parametrize("k,v", [
    (_rows(), _rows()),                                             # host tensors
    (torch.zeros(5, 8, 2, dtype=torch.bfloat16).transpose(1, 2), _rows()),  # strided rows
    (_rows(dtype=torch.float32), _rows(dtype=torch.float32)),
])
def test_a_refused_commit_changes_nothing(k, v):
    """No row stays reserved, and the step's weights are taken back, whatever refuses the commit."""
    store = _fresh()
    with pytest.raises((TypeError, ValueError)):
        store.commit([1], inputs._tree([(0, [(-1, 5)])], 0), None, k, v)
    assert store.length(1) == 0 and store.free_blocks() == 4 and not store._weighed
    assert store.mass[0].tolist() == list(range(48)) and not bool(store.mass[1].any())


def test_a_commit_that_the_library_refuses_gives_its_rows_back(monkeypatch):
    """The append's own refusal comes after the reservation: the rows and blocks are returned."""
    store = _fresh()
    monkeypatch.setattr(flide, "_ptr", lambda t: None)
    monkeypatch.setattr(flide, "_stream", lambda s=None: None)

    class Index:
        c = flide.TreeIndexC()

    with pytest.raises(flide.FlideError) as e:
        store.commit([1], inputs._tree([(0, [(-1, 5)])], 0), Index(), _rows(), _rows())
    assert e.value.code == flide.ERR_SHAPE
    assert store.length(1) == 0 and store.free_blocks() == 4 and not store._weighed
    assert store.lengths.tolist() == [0, 0] and not bool(store.mass[1].any())
