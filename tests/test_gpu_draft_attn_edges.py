"""Draft attention at the edges of its contract: every tile size at the most requests that a tile
takes, scales of zero, values that are not finite, one key that outweighs all others."""
import math

import numpy as np
import pytest
import torch

from tree_forked_decision_b200 import flide, inputs

import decode_helpers as dh
from gpu_helpers import build
from test_gpu_draft_attn import _cat, _check, _dev, _inputs, _wide

pytestmark = pytest.mark.gpu

KINDS = [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("f32", 64)]
# tokens of a request: with 4 heads to a group 4, 40, 100 and 200 query rows, a tile of each size
TOKENS = [1, 10, 25, 50]


def _draft(tree, x, hist, ds, scale):
    _, idx = build(tree)
    q, k, v = _dev(x)
    pk, pv = (_cat(h).cuda() for h in hist)
    out, lse = flide.draft_attn(q, k, v, idx, scale, past_k=pk, past_v=pv, descale=None if ds is None else ds.cuda())
    torch.cuda.synchronize()
    assert idx.status() == 0
    return out, lse


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("R", [967, 968, 1024])
def test_every_tile_with_many_requests(R, tokens, kind, d):
    """A call takes up to 2048 requests, whatever tile its rows ask for; every 41st request is checked."""
    rng = np.random.default_rng(R)
    past = rng.integers(0, 40, R).tolist()
    tree = inputs._tree([(n, [(-1, tokens)]) for n in past], 0)
    x, hist, ds = _inputs(tree, 4, 1, d, kind, 4)
    pools, table, slots, width = dh.scatter(hist, 16, rng)
    _, idx = build(tree)
    q, k, v = _dev(x)
    scale = 1 / math.sqrt(d)
    out, lse = flide.draft_attn_paged(q, k, v, idx, scale, pools[0].cuda(), pools[1].cuda(), table.cuda(), slots.cuda(),
                                      16, width, descale=None if ds is None else ds.cuda())
    torch.cuda.synchronize()
    assert idx.status() == 0
    some = list(range(0, R, 41)) + [R - 1]
    rows = torch.cat([torch.arange(r * tokens, (r + 1) * tokens) for r in some])
    _check(inputs._tree([(past[r], [(-1, tokens)]) for r in some], 0), [y[rows] for y in x],
           [[h[r] for r in some] for h in hist], ds, scale, out.cpu()[rows], lse.cpu()[rows], kind)


@pytest.mark.parametrize("kind,d", KINDS)
@pytest.mark.parametrize("tokens", TOKENS)
@pytest.mark.parametrize("scale", [0.0, 1e-45])
def test_scale_of_zero(scale, tokens, kind, d):
    """All scores are (nearly) equal: the mean of the values, whatever stands behind the history's end."""
    tree = inputs._tree([(n, [(-1, tokens)]) for n in (0, 1, 31, 33, 127, 128, 129, 300, 1025)], 0)
    x, hist, ds = _inputs(tree, 4, 1, d, kind, 5)
    out, lse = _draft(tree, x, hist, ds, scale)
    _check(tree, x, hist, ds, scale, out, lse, kind)


@pytest.mark.parametrize("tokens", TOKENS)
def test_factors_whose_product_vanishes(tokens):
    """descale[0] descale[1] below the least 32-bit number: as a scale of zero."""
    tree = inputs._tree([(n, [(-1, tokens)]) for n in (0, 1, 33, 129, 300)], 0)
    x, hist, _ = _inputs(tree, 4, 1, 128, "e4m3", 5)
    ds = torch.tensor([1e-30, 1e-30, 0.01])
    out, lse = _draft(tree, x, hist, ds, 0.1)
    _check(tree, x, hist, ds, 0.1, out, lse, "e4m3")


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("tokens", TOKENS)
def test_infinite_values_that_a_row_sees(tokens, kind, d):
    """An infinity among the values that a row sees, every weight above 0: infinite there, NaN where both
    signs meet or a NaN stands, and no other element is touched."""
    past = [1, 40, 129, 1000, 3001]
    tree = inputs._tree([(n, [(-1, tokens)]) for n in past], 0)
    x, hist, _ = _inputs(tree, 8, 2, d, kind, 6)
    for r, n in enumerate(past):
        v = hist[1][r]
        at = lambda share: min(n - 1, int(share * n))  # noqa: E731
        v[at(0.3), 0, 1] = math.inf
        v[at(0.99), 0, 2] = -math.inf
        v[at(0.6), 0, d - 1] = v[0, 0, d - 1] = math.inf   # twice, in different places
        if n > 1:
            v[at(0.2), 0, 5], v[n - 1, 0, 5] = math.inf, -math.inf
        if r % 2:
            v[at(0.5), 0, 7] = math.nan
    scale = 1 / math.sqrt(d)
    out, lse = _draft(tree, x, hist, None, scale)
    o, want, wv, peak, size = dh.attention(tree, *[y.double() for y in x], [h.double() for h in hist[0]],
                                           [h.double() for h in hist[1]], scale)
    got = out.double().cpu()
    assert torch.equal(got.isnan(), o.isnan())
    inf = o.isinf()
    assert bool(inf.any()) and torch.equal(got.isinf(), inf) and torch.equal(got[inf], o[inf])
    fine = o.isfinite()
    tol = dh.attention_tolerance(o, wv, peak, size, d, max(past) + tokens, out.dtype, 0.0 if kind == "f32" else 2.0 ** -8)
    assert bool(((got - o).abs()[fine] <= tol[fine]).all())
    assert bool(((lse.double().cpu() - want).abs() <= dh.lse_tolerance(want, size, d, max(past) + tokens)).all())


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("tokens", TOKENS)
def test_keys_that_are_all_nan(tokens, kind, d):
    """A history whose every key is NaN leaves no number in its rows, and the other requests alone."""
    tree = inputs._tree([(n, [(-1, tokens)]) for n in (50, 500, 60)], 0)
    x, hist, _ = _inputs(tree, 4, 1, d, kind, 7)
    scale = 1 / math.sqrt(d)
    was = _draft(tree, x, hist, None, scale)
    hist[0][1][:] = math.nan
    out, lse = _draft(tree, x, hist, None, scale)
    mid = slice(tokens, 2 * tokens)
    assert bool(out[mid].isnan().all()) and bool(lse[mid].isnan().all())
    for rows in (slice(0, tokens), slice(2 * tokens, 3 * tokens)):
        assert torch.equal(out[rows], was[0][rows]) and torch.equal(lse[rows], was[1][rows])


@pytest.mark.parametrize("spread", [0.0, 0.6])
@pytest.mark.parametrize("tokens", TOKENS)
def test_one_key_outweighs_each_other(tokens, spread):
    """e4m3: one key of weight 2^17 times each of 16384 others, which hold a ninth of the sum together (a
    first token that draws the attention).  A weight w of a row whose largest is L is off by at most
    max(2^-8 w, 2^-20 L), and by 2^-3 w from 2^-20 L on (two codes, e4m3 and e5m2, of w 2^6 / L)."""
    R, n, Hkv, d = 20, 16384, 8, 128
    g = torch.Generator().manual_seed(tokens)
    tree = inputs._tree([(n, [(-1, tokens)])] * R, 0)
    T = tree.T
    ds = torch.tensor([0.01, 0.01, 0.01])
    code = lambda y: (y / 0.01).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
    one = torch.ones(d)
    q = code(one.expand(T, 4 * Hkv, d) * (1 + 0.05 * torch.rand(T, 4 * Hkv, 1, generator=g)))
    hk = spread * torch.randn(n, Hkv, d, generator=g)
    hk[0] = 1.0
    hv = 1 + 0.25 * torch.rand(n, Hkv, d, generator=g)
    hv[0] = 0.0
    hk, hv = code(hk), code(hv)
    scale = 17 * math.log(2) / d
    k = code(-one.expand(T, Hkv, d))  # the stream's own keys: hardly any weight
    v = code(torch.ones(T, Hkv, d))
    bl, width = 128, n // 128
    table = torch.arange(width, dtype=torch.int32).repeat(R)  # every request reads the same blocks
    _, idx = build(tree)
    b = lambda y: y.contiguous().view(torch.uint8).cuda()  # noqa: E731
    out, lse = flide.draft_attn_paged(b(q), b(k), b(v), idx, scale, b(hk), b(hv), table.cuda(),
                                      torch.arange(R, dtype=torch.int32, device="cuda"), bl, width, descale=ds.cuda())
    torch.cuda.synchronize()
    assert idx.status() == 0
    f = lambda y: y.double().cuda() * float(ds[0])  # noqa: E731
    rows = torch.arange(0, T, max(1, T // 40))  # some tokens of all requests
    for h in range(0, 4 * Hkv, 5):
        kk, vv = f(hk[:, h // 4]), f(hv[:, h // 4])
        s = f(q[rows, h]) @ kk.T * scale
        w = torch.exp(s - s.amax(1, keepdim=True))
        own = torch.exp(-scale * d - s.amax(1)) * tokens * 1.2   # the stream's keys, at most
        total = w.sum(1, keepdim=True)
        o = (w / total) @ vv
        err = torch.where(w >= 2.0 ** -20, torch.minimum(w * 2.0 ** -3, torch.clamp(w * 2.0 ** -8, min=2.0 ** -20)), w)
        # 32-bit sums of as many terms; sizes of a score's products as in decode_helpers
        ds32 = (d + 4) * 2.0 ** -24 * float((f(q[rows, h]).abs() @ kk.abs().T * scale).max())
        rel = 2 * ds32 + 2.0 ** -20 + 2 * (n + tokens + 8) * 2.0 ** -24
        tol = 2.0 ** -8 * o + (err / total) @ vv + rel * o + 3 * (own / total[:, 0])[:, None] + 1e-9
        diff = (out[rows.cuda(), h].double() - o).abs()
        assert bool((diff <= tol).all()), float((diff / tol).max())
        if spread:  # weights that differ are rounded either way: the sum of 16384 is far closer
            assert float((diff / o).max()) < 2.0 ** -6


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (16, 4)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_long_paths(kind, Hq, Hkv):
    """Paths of more than 64 keys and more than 32 ancestors, with one, two and four heads to a warp of the join."""
    tree = inputs._tree([(n, [(-1, 150)] + [(i, 1 + i % 2) for i in range(45)]) for n in (0, 200)], 45)
    x, hist, ds = _inputs(tree, Hq, Hkv, 128, kind, 8)
    scale = 1 / math.sqrt(128)
    out, lse = _draft(tree, x, hist, ds, scale)
    _check(tree, x, hist, ds, scale, out, lse, kind)
