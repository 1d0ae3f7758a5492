"""Attention of small drafted trees over a long past (flide_draft_attn, packed and
paged) against the 64-bit form, with the elementwise bounds of decode_helpers."""
import math

import numpy as np
import pytest
import torch

from tree_forked_decision_b200 import flide, inputs

import decode_helpers as dh
from gpu_helpers import build

pytestmark = pytest.mark.gpu

TREES = {
    # one token on an empty history, one row of history, lengths around the kernels' tiles
    "one_token": lambda: inputs._tree([(0, [(-1, 1)])], 0),
    "one_row": lambda: inputs._tree([(1, [(-1, 1)])], 0),
    "edges": lambda: inputs._tree([(n, [(-1, 1), (0, 1), (0, 1)]) for n in
                                   (15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 257)], 1),
    # past only, root without tokens, requests without nodes, chains, deep and wide trees
    "odd_requests": lambda: inputs._tree([(70, []), (5, [(-1, 0), (0, 2), (0, 1)]), (0, []),
                                          (200, [(-1, 3), (0, 2), (1, 1), (2, 4), (0, 1), (4, 1)]), (0, [(-1, 4)]),
                                          (90, [(-1, 1)] + [(i, 1) for i in range(11)])], 11),
    "wide": lambda: inputs._tree([(700, [(-1, 4)] + [(max(0, i - 3), 1) for i in range(59)])], 59),
    # 16, 20 and 30 to 70 tokens a request: with 4 heads to a group tiles of 64, 128 and 256 rows
    "tile128": lambda: inputs._tree([(n, [(-1, 2)] + [(i // 2, 1) for i in range(14)]) for n in
                                     (0, 1, 127, 128, 129, 255, 256, 257, 383, 385, 2000)], 4),
    "tile256": lambda: inputs._tree([(n, [(-1, 3)] + [(i // 2, 1) for i in range(m)]) for n, m in
                                     ((0, 40), (1, 30), (127, 61), (128, 62), (129, 70), (513, 29), (3001, 61))], 6),
    "tile128_long": lambda: inputs._tree([(n, [(-1, 1)] + [(0, 1)] * 19) for n in (5100, 4900, 130, 5000)], 1),
    "tile80": lambda: inputs._tree([(n, [(-1, 1)] + [(i // 3, 1) for i in range(19)]) for n in
                                    (0, 1, 31, 33, 127, 129, 300, 1025)], 3),
    "long_one": lambda: inputs._tree([(5003, [(-1, 1), (0, 1), (1, 1)]), (3, [(-1, 2)])], 2),
    "many": lambda: inputs._tree([(int(n), [(-1, 1 + i % 3), (0, 1), (0, 2), (1, 1)]) for i, n in
                                  enumerate(np.random.default_rng(1).integers(0, 400, 37))], 2),
}
HEADS = [(4, 4), (16, 4), (8, 1), (12, 3), (5, 1), (40, 2), (14, 2), (129, 1), (100, 1)]


def _inputs(tree, Hq, Hkv, d, kind, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    T, past = tree.T, [int(p) for p in tree.past_len]
    x = [n(T, Hq, d), n(T, Hkv, d), n(T, Hkv, d)]
    hist = [[n(p, Hkv, d) for p in past] for _ in range(2)]
    if kind != "e4m3":
        t = {"bf16": torch.bfloat16, "f32": torch.float32}[kind]
        return [y.to(t) for y in x], [[y.to(t) for y in h] for h in hist], None
    ds = [0.01, 0.012, 0.009]
    code = lambda y, s: (y / s).clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
    return ([code(y, s) for y, s in zip(x, ds)],
            [[code(y, s) for y in h] for h, s in zip(hist, ds[1:])], torch.tensor(ds))


def _wide(y, s):
    return y.double() if s is None else y.double() * float(s)


def _check(tree, x, hist, ds, scale, got, lse, kind):
    d = x[0].shape[2]
    s = [None] * 3 if ds is None else ds
    o, want, wv, peak, size = dh.attention(tree, _wide(x[0], s[0]), _wide(x[1], s[1]), _wide(x[2], s[2]),
                                     [_wide(h, s[1]) for h in hist[0]], [_wide(h, s[2]) for h in hist[1]], scale)
    keys = int(tree.past_len.max()) + tree.T
    out = torch.float32 if kind == "f32" else torch.bfloat16
    # weights are rounded to bf16 before they multiply v; with e4m3 codes to half, or to an e4m3
    # code and its remainder's: each within half a step (2^-4) of what it stands for, 2^-8 together,
    # and never closer than half the least step, 2^-10, of weights scaled by 2^6
    w = {"f32": 0.0, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -8}[kind]
    tol = dh.attention_tolerance(o, wv, peak, size, d, keys, out, w, 2.0 ** -16 if kind == "e4m3" else 0.0)
    err = (got.double().cpu() - o).abs()
    assert got.dtype == out
    assert bool((err <= tol).all()), float((err / tol).max())
    err = (lse.double().cpu() - want).abs()
    assert bool((err <= dh.lse_tolerance(want, size, d, keys)).all()), float(err.max())


def _dev(x):
    return [y.cuda() for y in x]


def _cat(rows):
    return torch.cat([r.view(torch.uint8) if r.dtype == torch.float8_e4m3fn else r for r in rows])


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("case", sorted(TREES))
def test_packed(case, kind):
    tree = TREES[case]()
    for i, (Hq, Hkv) in enumerate(HEADS if case in ("edges", "odd_requests", "tile128") else HEADS[1:2]):
        for d in ([128] if kind == "e4m3" else [64, 128, 96, 256] if case == "odd_requests" else [128]):
            x, hist, ds = _inputs(tree, Hq, Hkv, d, kind, 3 + i)
            scale = 1 / math.sqrt(d)
            _, idx = build(tree)
            q, k, v = _dev(x)
            pk, pv = (_cat(h).cuda() for h in hist)
            out, lse = flide.draft_attn(q, k, v, idx, scale, past_k=pk, past_v=pv,
                                        descale=None if ds is None else ds.cuda())
            torch.cuda.synchronize()
            assert idx.status() == 0
            _check(tree, x, hist, ds, scale, out, lse, kind)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("block_rows", [16, 48, 128, 256])
@pytest.mark.parametrize("case", ["edges", "odd_requests", "wide", "tile128", "tile256", "tile80", "many"])
def test_paged_with_nan_behind_the_rows(case, block_rows, kind):
    """Rows of a block past a history's end hold NaN, and belong to nobody."""
    tree = TREES[case]()
    shapes = [(16, 4, 128)] + ([(16, 4, 64)] if kind == "bf16" else [])
    if case in ("edges", "many"):  # tiles with rows to spare; heads without a tcgen05 tile
        shapes += [(5, 1, 128), (21, 3, 128), (20, 1, 128), (130, 1, 128)] + ([] if kind == "e4m3" else [(8, 2, 64), (16, 1, 64)])
    for Hq, Hkv, d in shapes:
        x, hist, ds = _inputs(tree, Hq, Hkv, d, kind, 9)
        pools, table, slots, width = dh.scatter(hist, block_rows, np.random.default_rng(block_rows), fill=math.nan)
        _, idx = build(tree)
        q, k, v = _dev(x)
        scale = 1 / math.sqrt(d)
        out, lse = flide.draft_attn_paged(q, k, v, idx, scale, pools[0].cuda(), pools[1].cuda(), table.cuda(),
                                          slots.cuda(), block_rows, width, descale=None if ds is None else ds.cuda())
        torch.cuda.synchronize()
        assert idx.status() == 0
        _check(tree, x, hist, ds, scale, out, lse, kind)


@pytest.mark.parametrize("kind,d", [("bf16", 128), ("bf16", 64), ("e4m3", 128), ("f32", 64)])
@pytest.mark.parametrize("R", [1024, 1025, 2048])
def test_many_requests(R, kind, d):
    """One or two tokens a request, up to the most requests of a call."""
    rng = np.random.default_rng(R)
    tree = inputs._tree([(int(n), [(-1, 1 + i % 2)]) for i, n in enumerate(rng.integers(0, 40, R))], 0)
    x, hist, ds = _inputs(tree, 8, 2, d, kind, 4)
    pools, table, slots, width = dh.scatter(hist, 16, rng)
    _, idx = build(tree)
    q, k, v = _dev(x)
    scale = 1 / math.sqrt(d)
    out, lse = flide.draft_attn_paged(q, k, v, idx, scale, pools[0].cuda(), pools[1].cuda(), table.cuda(), slots.cuda(),
                                      16, width, descale=None if ds is None else ds.cuda())
    torch.cuda.synchronize()
    assert idx.status() == 0
    _check(tree, x, hist, ds, scale, out, lse, kind)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, torch.finfo(torch.bfloat16).min])
def test_a_masked_key_takes_no_part(bad):
    """A sibling branch full of NaN, infinities or the type's lowest value changes no bit of
    the other rows; rows behind the last token stay as they were."""
    tree = inputs._tree([(130, [(-1, 2), (0, 2), (0, 2), (1, 1)]), (40, [(-1, 1), (0, 1)])], 2)
    x, hist, _ = _inputs(tree, 16, 4, 128, "bf16", 4)
    q, k, v = _dev(x)
    pk, pv = (_cat(h).cuda() for h in hist)
    spare = 5
    pad = lambda y: torch.cat([y, torch.full((spare,) + y.shape[1:], math.nan, dtype=y.dtype, device="cuda")])  # noqa
    _, idx = build(tree, T=tree.T + spare)
    scale = 1 / math.sqrt(128)
    out = torch.full((tree.T + spare, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((tree.T + spare, 16), 7.0, device="cuda")
    flide.draft_attn(pad(q), pad(k), pad(v), idx, scale, past_k=pk, past_v=pv, out=out, lse=lse)
    assert bool((out[tree.T:] == 7).all()) and bool((lse[tree.T:] == 7).all())
    k2, v2 = k.clone(), v.clone()
    k2[4:6], v2[4:6] = bad, bad  # the second branch of request 0
    out2, lse2 = flide.draft_attn(pad(q), pad(k2), pad(v2), idx, scale, past_k=pk, past_v=pv)
    torch.cuda.synchronize()
    assert idx.status() == 0
    rows = [0, 1, 2, 3] + list(range(6, tree.T))
    assert torch.equal(out[rows], out2[rows]) and torch.equal(lse[rows], lse2[rows])
    _check(tree, x, hist, None, scale, out[:tree.T], lse[:tree.T], "bf16")


def test_equals_fork_attention():
    """The same keys as fork attention: both within the output's step of each other."""
    tree = inputs._tree([(1500, [(-1, 3), (0, 1), (0, 2), (2, 1)]), (640, [(-1, 1), (0, 4)])], 2)
    x, hist, _ = _inputs(tree, 16, 4, 128, "bf16", 5)
    q, k, v = _dev(x)
    pk, pv = (_cat(h).cuda() for h in hist)
    _, idx = build(tree)
    scale = 1 / math.sqrt(128)
    a = flide.fork_attn(q, k, v, idx, scale, past_k=pk, past_v=pv)
    b, _ = flide.draft_attn(q, k, v, idx, scale, past_k=pk, past_v=pv)
    torch.cuda.synchronize()
    assert float((a.float() - b.float()).norm() / a.float().norm()) < 2.0 ** -7


def test_device_errors():
    tree = inputs._tree([(200, [(-1, 1)]), (90, [(-1, 1)])], 0)
    x, hist, _ = _inputs(tree, 8, 2, 128, "bf16", 6)
    pools, table, slots, width = dh.scatter(hist, 64, np.random.default_rng(0))
    q, k, v = _dev(x)
    pk, pv = (p.cuda() for p in pools)
    call = lambda idx, tb, sl: flide.draft_attn_paged(q, k, v, idx, 0.1, pk, pv, tb.cuda(), sl.cuda(), 64, width)  # noqa
    hole = table.clone().view(-1, width)
    hole[int(slots[0]), 1] = -1
    far = table.clone().view(-1, width)
    far[int(slots[0]), 0] = pools[0].shape[0] // 64
    off = slots.clone()
    off[1] = table.numel() // width
    for tb, sl in ((hole.view(-1), slots), (far.view(-1), slots), (table, off)):
        _, idx = build(tree)
        call(idx, tb, sl)
        torch.cuda.synchronize()
        assert idx.status() == flide.ERR_INVALID
    _, idx = build(tree)
    flide.draft_attn(q, k, v, idx, 0.1, past_k=pk[:100].contiguous(), past_v=pv[:100].contiguous())
    torch.cuda.synchronize()
    assert idx.status() == flide.ERR_CAPACITY
    _, idx = build(tree)
    flide.draft_attn(q, k, v, idx, 0.1)
    torch.cuda.synchronize()
    assert idx.status() == flide.ERR_SHAPE


def test_a_past_that_is_too_long_is_refused():
    rows = (1 << 30) + 1
    tree = inputs._tree([(rows, [(-1, 1)]), (16, [(-1, 1)])], 0)
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v, pk, pv = (torch.randn(n, h, 64, generator=g, device="cuda").bfloat16()
                       for n, h in ((2, 2), (2, 1), (2, 1), (16, 1), (16, 1)))
    width = (1 << 26) + 1
    table = torch.zeros(2 * width, dtype=torch.int32, device="cuda")
    _, idx = build(tree)
    flide.draft_attn_paged(q, k, v, idx, 0.1, pk, pv, table, torch.arange(2, dtype=torch.int32, device="cuda"), 16,
                           width)
    torch.cuda.synchronize()
    assert idx.status() == flide.ERR_CAPACITY


@pytest.mark.parametrize("tokens", [1, 30])
def test_rows_past_32_bit_offsets(tokens):
    """The history's blocks behind 2^31 elements of a pool give the bits that they give at its start."""
    Hq, Hkv, d, bl, n_blocks = 32, 8, 128, 128, 16500
    assert n_blocks * bl * Hkv * d > 2 ** 31 + 8 * bl * Hkv * d
    tree = inputs._tree([(470, [(-1, tokens)]), (129, [(-1, tokens)])], 0)
    g = torch.Generator(device="cuda").manual_seed(3)
    T = tree.T
    q, k, v, hk, hv = (torch.randn(n, h, d, generator=g, device="cuda").bfloat16()
                       for n, h in ((T, Hq), (T, Hkv), (T, Hkv), (6 * bl, Hkv), (6 * bl, Hkv)))
    pk, pv = (torch.empty(n_blocks * bl, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    got = []
    for first in (0, n_blocks - 6):
        for pool, rows in ((pk, hk), (pv, hv)):
            pool[first * bl:(first + 6) * bl] = rows
        table = torch.tensor([4, 5, -1, -1, 0, 1, 2, 3], dtype=torch.int32, device="cuda")
        table = torch.where(table >= 0, table + first, table)
        _, idx = build(tree)
        out, lse = flide.draft_attn_paged(q, k, v, idx, 0.1, pk, pv, table, slots, bl, 4)
        mass = torch.zeros(2, 4 * bl, device="cuda")
        flide.history_mass(q, k, lse, idx, 0.1, pk, table, slots, bl, 4, mass)
        m1, status = mass.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        ln = torch.tensor([129 + tokens, 470 + tokens], dtype=torch.int32, device="cuda")
        kept = flide.history_evict(slots, ln, table, bl, 4, pk, pv, mass, 100, status, sinks=3, recent=9)
        torch.cuda.synchronize()
        assert idx.status() == 0 and int(status) == 0
        rows = [pool[(first + b) * bl:(first + b) * bl + 100].clone() for pool in (pk, pv) for b in (0, 4)]
        got.append([out, lse, m1, kept, mass] + rows)
        for i, r in enumerate(rows):  # the kept rows, moved to the front
            src = (hk, hv)[i // 2][(4 * bl if i % 2 else 0):]
            assert torch.equal(r, src[kept[i % 2].long()])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_two_streams_with_their_own_workspaces():
    tree = TREES["many"]()
    x, hist, _ = _inputs(tree, 16, 4, 128, "bf16", 8)
    pk, pv = (_cat(h).cuda() for h in hist)
    runs = []
    for i in range(2):
        _, idx = build(tree)
        q, k, v = _dev(x)
        runs.append((q * (1 + i), k, v, idx))
    want = [flide.draft_attn(*r, 0.1, past_k=pk, past_v=pv) for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [flide.draft_attn(*r, 0.1, past_k=pk, past_v=pv, stream=s) for r, s in zip(runs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
