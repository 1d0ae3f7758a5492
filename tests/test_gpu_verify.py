"""Verification of drafted trees against the rule as stated (decode_helpers.verify keeps and
normalises the residual itself); decisions and tokens have to be equal."""
import numpy as np
import pytest
import torch

from tree_forked_decision_b200 import flide, inputs

import decode_helpers as dh
from gpu_helpers import build

pytestmark = pytest.mark.gpu

TREES = {
    "root_only": lambda: inputs._tree([(0, [(-1, 1)]), (9, [(-1, 3)])], 0),
    "chain": lambda: inputs._tree([(0, [(-1, 2), (0, 5)]), (3, [(-1, 1), (0, 1), (1, 3)])], 2),
    "wide": lambda: inputs._tree([(0, [(-1, 1)] + [(0, 1)] * 40)] * 3, 1),
    "mixed": lambda: inputs._tree([(4, []), (0, [(-1, 0), (0, 2)]), (2, [(-1, 2), (0, 1), (0, 2), (1, 1), (1, 1),
                                                                       (2, 1), (4, 1), (4, 2)]), (0, [])] +
                                  [(0, [(-1, 1), (0, 1), (0, 1), (0, 1), (1, 1), (1, 1), (3, 1), (6, 1)])] * 6, 4),
}


def _draw(tree, V, seed, sampled, dtype, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    T = tree.T
    _, _, sees = dh.layout(tree)
    logits = sharp * torch.randn(T, V, generator=g)
    near = logits + 0.7 * torch.randn(T, V, generator=g)
    target, draft = torch.softmax(logits, 1).to(dtype), torch.softmax(near, 1).to(dtype)
    before = torch.tensor([s[-2] if len(s) > 1 else 0 for s in sees])
    if sampled:
        tok = torch.multinomial(draft.float()[before], 1, generator=g)[:, 0]
    else:
        best = draft.float().topk(min(V, 4), 1).indices
        rank = torch.zeros(T, dtype=torch.long)
        for b in set(before.tolist()):
            kids = [t for t in range(T) if len(sees[t]) > 1 and sees[t][-2] == b]
            for i, t in enumerate(kids):
                rank[t] = i % best.shape[1]  # beyond the best: repeats among siblings
        tok = best[before, rank]
    return (tok.to(torch.int32), target, draft if sampled else None, torch.rand(T, generator=g),
            torch.rand(tree.R, generator=g))


def _run(tree, tok, target, draft, u, un, **kw):
    _, idx = build(tree, **kw)
    n, nxt, path = flide.verify_draft(idx, tok.cuda(), target.cuda(), u.cuda(), un.cuda(),
                                      draft=None if draft is None else draft.cuda())
    torch.cuda.synchronize()
    return idx.status(), n.cpu().numpy(), nxt.cpu().numpy(), path.cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("V", [1, 5, 129, 1000, 8192])
@pytest.mark.parametrize("case", sorted(TREES))
def test_verify(case, V, sampled, dtype):
    tree = TREES[case]()
    for seed in range(4):
        args = _draw(tree, V, 31 * seed + V, sampled, dtype)
        status, n, nxt, path = _run(tree, *args)
        assert status == 0
        f = lambda x: None if x is None else x.float().numpy()  # noqa: E731
        want = dh.verify(tree, args[0].numpy(), f(args[1]), f(args[2]), f(args[3]), f(args[4]))
        assert np.array_equal(n, want[0]) and np.array_equal(nxt, want[1]) and np.array_equal(path, want[2])


def test_large_vocabulary():
    tree = TREES["mixed"]()
    args = _draw(tree, 150001, 5, True, torch.float32, sharp=4.0)
    status, n, nxt, path = _run(tree, *args)
    want = dh.verify(tree, *(x.numpy() for x in args))
    assert status == 0 and np.array_equal(n, want[0]) and np.array_equal(nxt, want[1]) and np.array_equal(path, want[2])


@pytest.mark.parametrize("sampled", [True, False])
def test_tokens_are_distributed_as_the_target(sampled):
    """4096 trees of one token with three drafted continuations: the token that follows (the first
    accepted one, or the next token) has the target's distribution.  Each of the 8 frequencies is a
    mean of 4096 trials, within 5 of its standard deviations (numbers are seeded)."""
    R, V = 4096, 8
    tree = inputs._tree([(0, [(-1, 1), (0, 1), (0, 1), (0, 1)])] * R, 1)
    g = torch.Generator().manual_seed(2)
    p = torch.softmax(torch.randn(V, generator=g), 0)
    q = torch.softmax(torch.randn(V, generator=g), 0)
    target = p.expand(4 * R, V).contiguous()
    if sampled:
        draft, tok = q.expand(4 * R, V).contiguous(), torch.multinomial(q, 4 * R, replacement=True, generator=g)
    else:
        draft, tok = None, q.topk(3).indices.new_tensor([0, *q.topk(3).indices.tolist()]).repeat(R)
    u, un = torch.rand(4 * R, generator=g), torch.rand(R, generator=g)
    status, n, nxt, path = _run(tree, tok.to(torch.int32), target, draft, u, un)
    assert status == 0
    first = path.reshape(R, 4)[:, 0]
    token = np.where(n > 0, tok.numpy()[np.maximum(first, 0)], nxt)
    freq = np.bincount(token, minlength=V) / R
    p = p.double().numpy()
    assert np.all(np.abs(freq - p) <= 5 * np.sqrt(p * (1 - p) / R))


def test_greedy_rows_and_edges():
    """One-hot target rows: the drafted token is accepted exactly if it is the target's; u = 0 and the
    largest u below 1; empty rows and rows with NaN, negative and infinite entries."""
    tree = inputs._tree([(0, [(-1, 1), (0, 1), (0, 1), (1, 1)])] * 2, 2)
    V = 300
    target = torch.zeros(tree.T, V)
    target[[0, 1, 2, 3], [7, 8, 9, 10]] = 1.0   # request 0: 7 is drafted second, 8 below the first
    target[[4, 5, 6, 7], [3, 299, 1, 299]] = 1.0
    tok = torch.tensor([0, 6, 7, 8, 0, 3, 2, 299], dtype=torch.int32)
    u = torch.full((tree.T,), 1 - 2.0 ** -24)
    status, n, nxt, path = _run(tree, tok, target, None, u, torch.tensor([0.0, 1 - 2.0 ** -24]))
    assert status == 0 and n.tolist() == [1, 2] and nxt.tolist() == [9, 299]
    assert path.tolist() == [2, -1, -1, -1, 5, 7, -1, -1]
    odd = target.clone()
    odd[0], odd[2] = 0.0, 0.0
    odd[4, :3] = torch.tensor([float("nan"), -2.0, 0.25])
    odd[4, 3] = 0.0
    status, n, nxt, path = _run(tree, tok, odd, None, torch.full((tree.T,), 0.5), torch.tensor([0.3, 0.9]))
    assert status == 0 and n.tolist() == [0, 0] and nxt.tolist() == [-1, 2]
    odd[4, 9] = float("inf")
    tok[5:7] = 0
    status, n, nxt, path = _run(tree, tok, odd, None, torch.full((tree.T,), 0.5), torch.tensor([0.3, 0.9]))
    assert status == 0 and nxt.tolist() == [-1, -1]


@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("V", [300, 1021, 40000])
def test_subnormal_and_negative_zero_entries(V, sampled):
    """-0 counts as 0 and a subnormal probability as its value: a row that holds nothing else is drawn from."""
    tree = inputs._tree([(0, [(-1, 1), (0, 1)])], 1)
    tiny = [11, 140, V - 3]
    target = torch.full((2, V), -0.0)
    target[0, tiny] = torch.tensor([1e-42, 3e-42, 2e-42])
    draft = torch.full((2, V), -0.0)
    draft[0, 5] = 1.0
    tok = torch.tensor([0, 5], dtype=torch.int32)
    for un, want in ((0.0, tiny[0]), (0.16, tiny[0]), (0.17, tiny[1]), (0.66, tiny[1]), (0.67, tiny[2]),
                     (1 - 2.0 ** -24, tiny[2])):
        status, n, nxt, path = _run(tree, tok, target, draft if sampled else None, torch.full((2,), 0.5),
                                    torch.tensor([un]))
        assert status == 0 and n.tolist() == [0] and nxt.tolist() == [want]


def test_bad_tokens_and_spare_rows():
    tree = TREES["mixed"]()
    tok, target, draft, u, un = _draw(tree, 64, 1, True, torch.float32)
    bad = tok.clone()
    bad[-1], bad[4] = 64, -1
    status, n, nxt, path = _run(tree, bad, target, draft, u, un)
    want = dh.verify(tree, *(x.numpy() for x in (bad, target, draft, u, un)))
    reached = status == flide.ERR_INVALID or (np.array_equal(n, want[0]) and status == 0)
    assert reached and np.array_equal(nxt, want[1])
    big = inputs._tree([(0, [(-1, 1)] + [(0, 1)] * 4096), (0, [(-1, 1)])], 1)
    uniform = torch.full((big.T, 4), 0.25)
    status, n, nxt, _ = _run(big, torch.zeros(big.T, dtype=torch.int32), uniform, None, torch.rand(big.T),
                             torch.tensor([0.1, 0.6]))
    assert status == flide.ERR_CAPACITY and n[0] == 0 and nxt[0] == -1
    _, idx = build(tree, T=tree.T + 4)
    path = torch.full((tree.T + 4,), 5, dtype=torch.int32, device="cuda")
    pad = lambda x: torch.cat([x, x[:4]]).cuda()  # noqa: E731
    flide.verify_draft(idx, pad(tok), pad(target), pad(u), un.cuda(), draft=pad(draft), path=path)
    assert path[tree.T:].tolist() == [5] * 4
