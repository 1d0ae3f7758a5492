"""History weight where a key holds infinities: a row whose every score is -inf gathers nothing, and no
other row's weight changes."""
import math

import numpy as np
import pytest
import torch

from tree_forked_decision_b200 import flide, inputs

import decode_helpers as dh
from gpu_helpers import build
from test_gpu_draft_attn import _dev, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("heads", [(2, 2), (8, 2), (5, 1), (24, 2)])
@pytest.mark.parametrize("root", [1, 3, 8])
def test_a_row_whose_scores_are_minus_infinity(root, heads, kind, d):
    Hq, Hkv = heads
    tree = inputs._tree([(200, [(-1, root), (0, 1)]), (33, [(-1, root)])], 1)
    x, hist, _ = _inputs(tree, Hq, Hkv, d, kind, 3)
    x[0][..., 5] = x[0][..., 5].abs() + 0.5  # every query's score with the rows below is -inf
    hist[0][0][17, :, 5] = -math.inf
    hist[0][1][32, :, 5] = -math.inf
    scale = 1 / math.sqrt(d)
    pools, table, slots, width = dh.scatter(hist, 16, np.random.default_rng(2), extra=root)
    pk, pv, table, slots = pools[0].cuda(), pools[1].cuda(), table.cuda(), slots.cuda()
    _, idx = build(tree)
    q, k, v = _dev(x)
    out, lse = flide.draft_attn_paged(q, k, v, idx, scale, pk, pv, table, slots, 16, width)
    mass = torch.zeros((table.numel() // width, width * 16), device="cuda")
    flide.history_mass(q, k, lse, idx, scale, pk, table, slots, 16, width, mass)
    torch.cuda.synchronize()
    assert idx.status() == 0 and bool(out.isfinite().all()) and bool(lse.isfinite().all())
    want = dh.mass_of(tree, x[0], x[1], hist[0], lse.cpu(), scale)
    size = 2 * d * scale * 20  # products of a score, at most (rows without the infinity): |q|, |k| below 5
    rel = (d + 4) * 2.0 ** -24 * size + 2.0 ** -20 + 2.0 ** -23 * float(lse.abs().max()) + 2.0 ** -24 * Hq * 64
    got = mass.cpu().double()
    for r, row in enumerate((17, 32)):
        n = want[r].shape[0]
        mine = got[int(slots[r]), :n]
        assert float(want[r][row]) == 0 and float(mine[row]) == 0
        assert bool(((mine - want[r]).abs() <= rel * want[r] + 1e-12).all())
