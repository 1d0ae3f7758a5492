"""Verification past its shared-memory tables: many drafted tokens, more continuations than are tried,
vocabularies whose segments are longer than a warp's step; what a bad token leaves."""
import numpy as np
import pytest
import torch

from tree_forked_decision_b200 import flide, inputs

import decode_helpers as dh
from test_gpu_verify import TREES, _draw, _run

pytestmark = pytest.mark.gpu


def _same(got, want):
    return all(np.array_equal(a, b) for a, b in zip(got, want))


def _want(tree, *args):
    return dh.verify(tree, *(None if x is None else x.float().numpy() if x.is_floating_point() else x.numpy()
                             for x in args))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("stop", [200, 511, 512, 513, 700])
def test_more_drafted_tokens_than_are_held(stop, sampled, dtype):
    """A path of up to 700 tokens, every one of them accepted up to `stop`, among 912 drafted ones."""
    tree = inputs._tree([(0, [(-1, 2), (0, 300), (1, 1), (1, 400)] + [(2, 1)] * 10 + [(3, 1)] * 200), (0, [(-1, 1), (0, 1)])],
                        3)
    tok, target, draft, u, un = _draw(tree, 40, 3, sampled, dtype)
    if draft is not None:
        target = draft.clone()  # (p = q: any u is accepted)
    u[2:2 + stop] = 0.0
    if stop < 700:
        target[1 + stop] = target[1 + stop].roll(1)
    # the node of 400 tokens follows another child, which is refused
    tok[302] = int(target[301].float().argmin())
    target[301, int(tok[302])] = 0.0
    if draft is not None:
        tok[303] = int(draft[301].float().argmax())
    status, *got = _run(tree, tok, target, draft, u, un)
    want = _want(tree, tok, target, draft, u, un)
    assert status == 0 and _same(got, want)


@pytest.mark.parametrize("kids", [1023, 1024, 1025, 1100])
@pytest.mark.parametrize("sampled", [True, False])
def test_more_continuations_than_are_tried(sampled, kids):
    """1024 continuations of a token are tried; beyond them the call reports it and draws the next token from what
    the tried ones left."""
    V = 2048
    tree = inputs._tree([(0, [(-1, 1)] + [(0, 1)] * kids), (0, [(-1, 1), (0, 1)])], 1)
    g = torch.Generator().manual_seed(kids)
    T = tree.T
    target, draft = torch.rand(T, V, generator=g), torch.rand(T, V, generator=g)
    tok = torch.arange(-1, T - 1, dtype=torch.int32) % V
    if sampled:
        target[0, :1200] = 0.0  # what is drafted is refused
    target, draft = target / target.sum(1, keepdim=True), draft / draft.sum(1, keepdim=True)
    u = torch.full((T,), 1 - 2.0 ** -24)
    un = torch.tensor([0.37, 0.5])
    status, n, nxt, path = _run(tree, tok, target, draft if sampled else None, u, un)
    tried = min(kids, 1024)
    first = inputs._tree([(0, [(-1, 1)] + [(0, 1)] * tried), (0, [(-1, 1), (0, 1)])], 1)
    keep = torch.tensor(list(range(1 + tried)) + [T - 2, T - 1])
    want = _want(first, tok[keep], target[keep], draft[keep] if sampled else None, u[keep], un)
    assert status == (flide.ERR_CAPACITY if kids > 1024 else 0)
    assert np.array_equal(n, want[0]) and np.array_equal(nxt, want[1])
    assert want[0][0] == 0 and bool((path[:1 + kids] == -1).all())


@pytest.mark.parametrize("R,V,sampled", [(1, 2300003, True), (1, 2300000, False), (38, 1060000, False), (38, 1060001, True)])
def test_long_segments(R, V, sampled):
    """Vocabularies past 2^20 entries (16 blocks to a tree) and past 2^20 with 8 blocks to each of more trees."""
    g = torch.Generator().manual_seed(R)
    tree = inputs._tree([(0, [(-1, 1), (0, 1)] if R == 1 else [(-1, 1)])] * R, 1 if R == 1 else 0)
    T = tree.T
    target = torch.rand(T, V, generator=g) ** 4
    target /= target.sum(1, keepdim=True)
    draft = None
    tok = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    u = torch.full((T,), 0.9999)
    if sampled:
        draft = target.roll(7, 1)
        tok[1] = int(draft[0].argmax())  # (T of 2: refused, its residual is drawn from)
    un = torch.linspace(0, 1 - 2.0 ** -24, R) if R > 1 else torch.tensor([0.731])
    status, *got = _run(tree, tok, target, draft, u, un)
    assert status == 0 and _same(got, _want(tree, tok, target, draft, u, un))


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("token", [-1, 64, 2 ** 31 - 1, -2 ** 31])
def test_a_bad_token_is_reported_and_passed_over(token, sampled):
    """A drafted token outside the vocabulary that the walk reaches: status INVALID; it is never accepted, and the
    accepted tokens, the next one and the path are those of the others."""
    tree = TREES["mixed"]()
    for seed in range(4):
        tok, target, draft, u, un = _draw(tree, 64, seed, sampled, torch.float32)
        first = int(np.cumsum([0, *tree.seg_len])[tree.req_node_ptr[2] + 1])  # the first child of request 2's root
        tok[first] = token
        status, *got = _run(tree, tok, target, draft, u, un)
        assert status == flide.ERR_INVALID
        assert _same(got, _want(tree, tok, target, draft, u, un))
