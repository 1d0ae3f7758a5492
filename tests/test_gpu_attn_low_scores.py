"""Fork attention where every score is far below 0: the row's maximum is that of its own scores."""
import math

import pytest
import torch

from tree_forked_decision_b200 import flide, inputs

import decode_helpers as dh
from gpu_helpers import build
from test_gpu_draft_attn import _cat, _check, _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("low", [-40.0, -300.0, -3000.0])
@pytest.mark.parametrize("heads", [(4, 4), (16, 4)])
def test_low_scores(heads, low):
    Hq, Hkv, d = *heads, 128
    g = torch.Generator().manual_seed(1)
    tree = inputs._tree([(300, [(-1, 200), (0, 40), (0, 70), (1, 3)]), (0, [(-1, 130), (0, 1)])], 2)
    scale = 1 / math.sqrt(d)
    # q along the first axis, k against it: scores low + noise of a unit
    def rows(n, H, first):
        y = torch.randn(n, H, d, generator=g)
        y[..., 0] = first
        return y.bfloat16()
    x = [rows(tree.T, Hq, 4.0), rows(tree.T, Hkv, low / 4 / scale), rows(tree.T, Hkv, 1.0)]
    hist = [[rows(int(p), Hkv, f) for p in tree.past_len] for f in (low / 4 / scale, 1.0)]
    _, idx = build(tree)
    q, k, v = _dev(x)
    out = flide.fork_attn(q, k, v, idx, scale, past_k=_cat(hist[0]).cuda(), past_v=_cat(hist[1]).cuda())
    torch.cuda.synchronize()
    assert idx.status() == 0
    _, lse, _, _, _ = dh.attention(tree, *x, *hist, scale)
    _check(tree, x, hist, None, scale, out, lse, "bf16")
