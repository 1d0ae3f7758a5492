"""Fork attention where every score is far below 0, or 0: the row's maximum is that of its own scores, and
masked keys weigh nothing."""
import math

import pytest
import torch

from tree_forked_decision_b200 import flide, inputs

import decode_helpers as dh
from gpu_helpers import build
from test_gpu_draft_attn import _cat, _check, _dev, _inputs

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


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("heads", [(4, 4), (16, 4)])
def test_scale_of_zero(heads, kind):
    """The mean of the values that a row sees, in tiles with masked keys too."""
    tree = inputs._tree([(300, [(-1, 200), (0, 40), (0, 70), (1, 3)]), (0, [(-1, 130), (0, 1)]), (128, [(-1, 1)])], 2)
    x, hist, ds = _inputs(tree, *heads, 128, kind, 2)
    _, idx = build(tree)
    past = dict(past_k=_cat(hist[0]).cuda(), past_v=_cat(hist[1]).cuda())
    if kind == "e4m3":
        q, k, v = (y.view(torch.uint8).cuda() for y in x)
        out = flide.fork_attn_fp8(q, k, v, idx, 0.0, ds.cuda(), **past)
    else:
        out = flide.fork_attn(*_dev(x), idx, 0.0, **past)
    torch.cuda.synchronize()
    assert idx.status() == 0
    f = [1.0] * 3 if ds is None else ds.tolist()
    o, _, _, _, _ = dh.attention(tree, *(y.double() * s for y, s in zip(x, f)), [h.double() * f[1] for h in hist[0]],
                                 [h.double() * f[2] for h in hist[1]], 0.0)
    # equal weights are 2^6 or 1, exact in every type: the output's rounding and 32-bit sums
    keys = 300 + tree.T
    size = max(float(h.double().abs().max()) * f[2] for h in (x[2], *hist[1]) if h.numel())
    tol = dh.step(out.dtype) * o.abs() + 4 * (keys + 8) * 2.0 ** -24 * size
    assert bool(((out.double().cpu() - o).abs() <= tol).all())
