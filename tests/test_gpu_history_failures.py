"""What a refused call leaves of a HistoryStore: its weights, lengths and blocks as they were."""
import pytest
import torch

from tree_forked_decision_b200 import flide, inputs
from tree_forked_decision_b200.history import HistoryStore

pytestmark = pytest.mark.gpu

Hq, Hkv, d = 8, 2, 64


def _step(store, slots, roots, seed):
    """(tree, index, k, v) of a step whose roots have these tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    tree = inputs._tree([(store.length(s) if s >= 0 else 0, [(-1, m)]) for s, m in zip(slots, roots)], 0)
    dt = flide.DeviceTree(*tree.arrays(), max_depth=0)
    idx = flide.TreeIndex(dt.R, dt.N, dt.T, 0)
    flide.tree_build(dt, idx)
    q, k, v = n(tree.T, Hq, d), n(tree.T, Hkv, d), n(tree.T, Hkv, d)
    _, lse = store.draft_attn(q, k, v, idx, 0.1, slots)
    store.accumulate_mass(q, k, lse, idx, 0.1, slots)
    return tree, idx, k, v


def _store(n_blocks=6):
    """Slots 2 and 0 with 40 and 20 rows: 5 blocks."""
    store = HistoryStore(n_blocks=n_blocks, block_rows=16, max_requests=3, max_blocks=4, Hkv=Hkv, d=d)
    slots = [2, 0]
    tree, idx, k, v = _step(store, slots, [40, 20], 1)
    store.commit(slots, tree, idx, k, v)
    return store, slots


def test_a_refused_commit_takes_its_weights_back():
    """Blocks run out: the weights of the step are not counted, so its retry counts them once."""
    store, slots = _store()
    before, held = store.mass.clone(), [store.length(s) for s in range(3)]
    tree, idx, k, v = _step(store, slots, [10, 30], 2)
    assert not torch.equal(store.mass, before)
    with pytest.raises(flide.FlideError) as e:
        store.commit(slots, tree, idx, k, v)
    assert e.value.code == flide.ERR_CAPACITY
    assert torch.equal(store.mass, before) and [store.length(s) for s in range(3)] == held
    tree, idx, k, v = _step(store, slots, [10, 8], 3)
    once = store.mass.clone()
    store.commit(slots, tree, idx, k, v)
    assert torch.equal(store.mass, once)
    # the same step on a store that was never refused
    other, _ = _store()
    tree, idx, k, v = _step(other, slots, [10, 8], 3)
    assert torch.equal(other.mass, once)


def test_only_the_refused_slots_are_taken_back():
    """Two batches weigh their slots, then both commit; the one that is refused loses its own weights only."""
    store, _ = _store(n_blocks=5)
    before = store.mass.clone()
    a = _step(store, [0], [4], 4)
    b = _step(store, [2], [24], 5)
    both = store.mass.clone()
    with pytest.raises(flide.FlideError):
        store.commit([2], *b)
    assert torch.equal(store.mass[2], before[2]) and torch.equal(store.mass[0], both[0])
    store.commit([0], *a)
    assert torch.equal(store.mass[0], both[0]) and store.length(0) == 24
    # a later refusal does not bring back what was committed
    with pytest.raises(flide.FlideError):
        store.commit([0], *_step(store, [0], [20], 6))
    assert torch.equal(store.mass[0], both[0])


def test_released_and_evicted_slots_are_not_brought_back():
    store, slots = _store()
    _, idx, k, _ = _step(store, slots, [10, 30], 7)
    store.release(2)
    store.evict([0], 8, sinks=1, recent=2)
    after = store.mass.clone()
    rows = k.new_zeros(91, Hkv, d)
    with pytest.raises(flide.FlideError):
        store.commit([0, 2], inputs._tree([(0, [(-1, 90)]), (0, [(-1, 1)])], 0), idx, rows, rows)
    assert torch.equal(store.mass, after) and not bool(store.mass[2].any())


@pytest.mark.parametrize("bad", [3, 100])
def test_slots_that_are_none_of_the_store(bad):
    store, slots = _store()
    before = (store.mass.clone(), store.pool_k.clone(), store.lengths.clone())
    with pytest.raises(flide.FlideError) as e:
        store.evict([0, bad], 8)
    assert e.value.code == flide.ERR_INVALID
    with pytest.raises(flide.FlideError) as e:
        store.accumulate_mass(None, None, None, None, 0.1, [bad, 0])
    assert e.value.code == flide.ERR_INVALID
    torch.cuda.synchronize()
    assert torch.equal(store.mass, before[0]) and torch.equal(store.pool_k, before[1])
    assert torch.equal(store.lengths, before[2]) and int(store.status) == 0
