"""Attention weight of history rows (flide_history_mass) and eviction by it."""
import math

import numpy as np
import pytest
import torch

from tree_forked_decision_b200 import flide, inputs

import decode_helpers as dh
from gpu_helpers import build
from test_gpu_draft_attn import _dev, _inputs, _wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
@pytest.mark.parametrize("heads", [(4, 4), (16, 4), (32, 8), (8, 1), (12, 3), (40, 2)])
@pytest.mark.parametrize("block_rows", [16, 48, 128])
def test_mass(block_rows, heads, kind):
    """A weight is exp of (score - lse), off by what both are off (the attention's bound on a score,
    and the 32-bit lse given here exactly rounded); a row's sum adds terms of one sign, so its error
    is at most the terms' plus one rounding per term."""
    Hq, Hkv = heads
    d = 128 if kind == "e4m3" or Hq == 16 else 64 if Hq == 4 else 96 if Hq == 12 else 128
    tree = inputs._tree([(300, [(-1, 2), (0, 2), (0, 1)]), (0, [(-1, 5)]), (17, [(-1, 0), (0, 1)]), (1, [(-1, 1)]),
                         (0, []), (127, [(-1, 37)]), (64, [(-1, 3)])], 1)
    x, hist, ds = _inputs(tree, Hq, Hkv, d, kind, 11)
    s = [None] * 3 if ds is None else ds
    scale = 1 / math.sqrt(d)
    wide = [_wide(y, z) for y, z in zip(x, s)]
    pk, pv = [_wide(h, s[1]) for h in hist[0]], [_wide(h, s[2]) for h in hist[1]]
    _, lse, _, _, size = dh.attention(tree, *wide, pk, pv, scale)
    lse = lse.float()
    pools, table, slots, width = dh.scatter(hist[:1], block_rows, np.random.default_rng(1), extra=40, fill=math.nan)
    g = torch.Generator().manual_seed(3)
    old = torch.rand((table.numel() // width, width * block_rows), generator=g) * 50
    slots = slots.clone()
    gone = int(slots[6])
    slots[6] = -1  # keeps no history
    past = np.array(tree.past_len)
    past[6] = 0
    tree2 = inputs._tree([(int(past[r]), list(zip(tree.parent[tree.req_node_ptr[r]:tree.req_node_ptr[r + 1]].tolist(),
                                                  tree.seg_len[tree.req_node_ptr[r]:tree.req_node_ptr[r + 1]].tolist())))
                          for r in range(tree.R)], 1)
    _, idx = build(tree2)
    q, k, _ = _dev(x)
    out = torch.full_like(old, -3.0).cuda()
    args = (q, k, lse.cuda(), idx, scale, pools[0].cuda(), table.cuda(), slots.cuda(), block_rows, width)
    flide.history_mass(*args, old.cuda(), mass_out=out, descale=None if ds is None else ds.cuda())
    here = old.cuda()
    flide.history_mass(*args, here, descale=None if ds is None else ds.cuda())
    torch.cuda.synchronize()
    assert idx.status() == 0
    out, here = out.cpu(), here.cpu()
    want = dh.mass_of(tree, wide[0], wide[1], pk, lse, scale)
    rel = (d + 4) * 2.0 ** -24 * size + 2.0 ** -20 + 2.0 ** -23 * float(lse.abs().max()) + 2.0 ** -24 * Hq * 64
    touched = torch.zeros_like(out, dtype=torch.bool)
    for r in range(tree.R):
        if want[r] is None or int(slots[r]) < 0:
            continue
        n, total, sl = int(past[r]), want[r].shape[0], int(slots[r])
        base = old[sl, :total].double().clone()
        base[n:] = 0
        full = base + want[r]
        err = (out[sl, :total].double() - full).abs()
        assert bool((err <= rel * want[r] + 2.0 ** -24 * full + 1e-12).all()), float((err / full).max())
        touched[sl, :total] = True
    assert bool((out[~touched] == -3).all())
    assert torch.equal(here[touched], out[touched]) and torch.equal(here[~touched], old[~touched])
    assert gone >= 0


def test_mass_sums_to_the_tokens_and_heads():
    """What a root token gives its history and its root adds up to 1 for each head (no branches are
    among its keys): with lse of the draft attention itself."""
    tree = inputs._tree([(900, [(-1, 3), (0, 2)]), (33, [(-1, 1)])], 1)
    x, hist, _ = _inputs(tree, 16, 4, 128, "bf16", 2)
    pools, table, slots, width = dh.scatter(hist, 64, np.random.default_rng(2), extra=8)
    pk, pv = (p.cuda() for p in pools)
    q, k, v = _dev(x)
    _, idx = build(tree)
    scale = 1 / math.sqrt(128)
    _, lse = flide.draft_attn_paged(q, k, v, idx, scale, pk, pv, table.cuda(), slots.cuda(), 64, width)
    mass = torch.zeros((table.numel() // width, width * 64), device="cuda")
    flide.history_mass(q, k, lse, idx, scale, pk, table.cuda(), slots.cuda(), 64, width, mass)
    torch.cuda.synchronize()
    assert idx.status() == 0
    got = mass.double().sum(1).cpu()[slots.long()]
    # 32-bit weights and lse: within 1e-5 of their count
    assert np.allclose(got.numpy(), [3 * 16, 16], rtol=1e-5)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_mass_of_many_requests(kind):
    """The most requests of a call, each with one group of rows or two."""
    R, Hq, Hkv, d = 2048, 8, 2, 128
    rng = np.random.default_rng(2)
    tree = inputs._tree([(int(n), [(-1, 1 + i % 2)]) for i, n in enumerate(rng.integers(0, 20, R))], 0)
    x, hist, ds = _inputs(tree, Hq, Hkv, d, kind, 8)
    s = [None] * 3 if ds is None else ds
    scale = 1 / math.sqrt(d)
    pk = [_wide(h, s[1]) for h in hist[0]]
    _, lse, _, _, size = dh.attention(tree, *[_wide(y, z) for y, z in zip(x, s)], pk,
                                      [_wide(h, s[2]) for h in hist[1]], scale)
    lse = lse.float()
    pools, table, slots, width = dh.scatter(hist[:1], 16, rng, extra=2)
    _, idx = build(tree)
    q, k, _ = _dev(x)
    mass = torch.zeros((table.numel() // width, width * 16), device="cuda")
    flide.history_mass(q, k, lse.cuda(), idx, scale, pools[0].cuda(), table.cuda(), slots.cuda(), 16, width, mass,
                       descale=None if ds is None else ds.cuda())
    torch.cuda.synchronize()
    assert idx.status() == 0
    want = dh.mass_of(tree, _wide(x[0], s[0]), _wide(x[1], s[1]), pk, lse, scale)
    rel = (d + 4) * 2.0 ** -24 * size + 2.0 ** -20 + 2.0 ** -23 * float(lse.abs().max()) + 2.0 ** -24 * Hq * 64
    got = mass.cpu().double()
    for r in range(R):
        n = want[r].shape[0]
        err = (got[int(slots[r]), :n] - want[r]).abs()
        assert bool((err <= rel * want[r] + 2.0 ** -24 * want[r] + 1e-12).all())
        assert not bool(got[int(slots[r]), n:].any())


def test_mass_errors():
    tree = inputs._tree([(200, [(-1, 1)]), (90, [(-1, 60)])], 0)
    x, hist, _ = _inputs(tree, 8, 2, 128, "bf16", 6)
    pools, table, slots, width = dh.scatter(hist[:1], 64, np.random.default_rng(0))
    q, k, _ = _dev(x)
    lse = torch.zeros(tree.T, 8, device="cuda")
    n_slots = table.numel() // width

    def status(tb, sl, w=width):
        _, idx = build(tree)
        flide.history_mass(q, k, lse, idx, 0.1, pools[0].cuda(), tb.cuda(), sl.cuda(), 64, w,
                           torch.zeros((n_slots, w * 64), device="cuda"))
        torch.cuda.synchronize()
        return idx.status()

    hole = table.clone().view(-1, width)
    hole[int(slots[0]), 1] = -1
    off = slots.clone()
    off[1] = n_slots
    assert status(hole.view(-1), slots) == flide.ERR_INVALID
    assert status(table, off) == flide.ERR_INVALID
    assert status(table, slots) == 0
    grown = inputs._tree([(200, [(-1, 1)]), (200, [(-1, 60)])], 0)  # 200 + 60 rows do not fit 4 blocks of 64
    _, idx = build(grown)
    assert width == 4
    full = table.clone().view(-1, width)
    full[int(slots[1])] = full[int(slots[0])]
    flide.history_mass(q, k, lse, idx, 0.1, pools[0].cuda(), full.view(-1).cuda(), slots.cuda(), 64, width,
                       torch.zeros((n_slots, width * 64), device="cuda"))
    torch.cuda.synchronize()
    assert idx.status() == flide.ERR_CAPACITY
    past = inputs._tree([(200, [(-1, 1)]), (300, [(-1, 60)])], 0)  # nor does the past alone: no weight is written
    _, idx = build(past)
    before = torch.rand((n_slots, width * 64), device="cuda")
    mass = before.clone()
    flide.history_mass(q, k, lse, idx, 0.1, pools[0].cuda(), full.view(-1).cuda(), slots.cuda(), 64, width, mass)
    torch.cuda.synchronize()
    assert idx.status() == flide.ERR_CAPACITY
    assert torch.equal(mass[int(slots[1])], before[int(slots[1])])


# ---- eviction ----

SHAPES = [  # lengths, budget, sinks, recent, block rows, (Hkv, d), type
    ([5], 4, 0, 0, 16, (1, 8), torch.bfloat16),
    ([1, 0, 2], 1, 1, 0, 16, (2, 64), torch.float32),
    ([300, 17, 128, 129], 128, 4, 20, 16, (4, 128), torch.bfloat16),
    ([1000, 999, 40], 40, 0, 40, 48, (3, 64), torch.uint8),
    ([2500, 1024, 1025, 3000], 1025, 5, 0, 128, (2, 64), torch.bfloat16),
    ([5000], 100, 60, 40, 64, (1, 16), torch.bfloat16),
    ([4099, 4097], 4096, 1, 1, 256, (5, 16), torch.float32),
]


def _values(kind, n, g):
    m = torch.exp(3 * torch.randn(n, generator=g))
    if kind == "ties":
        m = torch.randint(0, 4, (n,), generator=g).float()
    elif kind == "equal":
        m[:] = 0.5
    elif kind == "odd":  # zeros of both signs, negative, tiny, infinite, NaN
        pick = torch.randint(0, 9, (n,), generator=g)
        m = torch.tensor([0.0, -0.0, -1.5, 1e-42, math.inf, -math.inf, math.nan, 2.0, 1e30])[pick]
    return m


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"{s[0][0]}to{s[1]}" for s in SHAPES])
def test_evict(shape, kind, in_place):
    lens, budget, sinks, recent, bl, (Hkv, d), t = shape
    g = torch.Generator().manual_seed(len(kind) + lens[0])
    rows = [[(torch.randint(0, 255, (n, Hkv, d), generator=g).to(t) if t == torch.uint8 else
              torch.randn(n, Hkv, d, generator=g).to(t)) for n in lens] for _ in range(2)]
    pools, table, slots, width = dh.scatter(rows, bl, np.random.default_rng(lens[0]))
    cap, n_slots = width * bl, table.numel() // width
    mass = torch.stack([_values(kind, cap, g) for _ in range(n_slots)])
    hist = torch.full((n_slots,), -5, dtype=torch.int32)  # an unused slot is not looked at
    hist[slots.long()] = torch.tensor(lens, dtype=torch.int32)
    pk, pv = (p.cuda() for p in pools)
    tb, m0, status = table.cuda(), mass.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {}
    if not in_place:
        need = [-(-min(n, budget) // bl) for n in lens]
        to = np.full((n_slots, width), -1, np.int32)
        ids = np.random.default_rng(3).permutation(sum(need) + 1)
        for r, c in enumerate(need):
            to[int(slots[r]), :c], ids = ids[:c], ids[c:]
        dst = [torch.full(((sum(need) + 1) * bl, Hkv, d), 3, dtype=t, device="cuda") for _ in range(2)]
        kw = dict(dst_k=dst[0], dst_v=dst[1], dst_table=torch.from_numpy(to.ravel()).cuda(),
                  mass_out=torch.full_like(m0, 77.0))
        before = (pk.clone(), pv.clone(), m0.clone())
    kept = flide.history_evict(slots.cuda(), hist.cuda(), tb, bl, width, pk, pv, m0, budget, status, sinks=sinks,
                               recent=recent, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    if not in_place:
        assert torch.equal(pk, before[0]) and torch.equal(pv, before[1])
        assert torch.equal(m0.view(torch.int32), before[2].view(torch.int32))
    out = (pk, pv) if in_place else dst
    where = table.view(-1, width) if in_place else torch.from_numpy(to)
    mo = (m0 if in_place else kw["mass_out"]).cpu()
    for r, n in enumerate(lens):
        sl = int(slots[r])
        want = dh.keep_rows(mass[sl].tolist(), n, budget, sinks, recent)
        assert kept[r].cpu().tolist() == want + [-1] * (budget - len(want))
        j = torch.arange(len(want))
        at = where[sl][j // bl].long() * bl + j % bl
        for got, src in zip(out, rows):
            assert torch.equal(got.cpu()[at], src[r][want])
        assert torch.equal(mo[sl, :len(want)].view(torch.int32), mass[sl][want].view(torch.int32))


def test_evict_refuses_on_the_device():
    lens, bl = [40, 50, 30], 16
    g = torch.Generator().manual_seed(0)
    rows = [[torch.randn(n, 2, 64, generator=g) for n in lens] for _ in range(2)]
    pools, table, slots, width = dh.scatter(rows, bl, np.random.default_rng(0))
    n_slots = table.numel() // width
    hist = torch.zeros(n_slots, dtype=torch.int32)
    hist[slots.long()] = torch.tensor(lens, dtype=torch.int32)
    mass = torch.rand(n_slots, width * bl, generator=g)

    def run(sl, ln, tb=table):
        pk, pv, status = pools[0].cuda(), pools[1].cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
        kept = flide.history_evict(sl.cuda(), ln.cuda(), tb.cuda(), bl, width, pk, pv, mass.cuda(), 20, status)
        torch.cuda.synchronize()
        return int(status), kept.cpu(), pk.cpu()

    twice = slots.clone()
    twice[2] = twice[0]
    code, kept, pk = run(twice, hist)
    assert code == flide.ERR_INVALID and bool((kept[[0, 2]] == -1).all()) and bool((kept[1] >= 0).all())
    at = table.view(-1, width)[int(slots[0])][torch.arange(40) // bl].long() * bl + torch.arange(40) % bl
    assert torch.equal(pk[at], rows[0][0])  # left as it was
    off = slots.clone()
    off[1] = n_slots
    assert run(off, hist)[0] == flide.ERR_INVALID
    for n in (-1, width * bl + 1):
        bad = hist.clone()
        bad[int(slots[0])] = n
        assert run(slots, bad)[0] == flide.ERR_INVALID
    hole = table.clone().view(-1, width)
    hole[int(slots[1])] = -1
    assert run(slots, hist, hole.view(-1))[0] == flide.ERR_INVALID
    none = torch.full_like(slots, -1)
    code, kept, pk = run(none, hist)
    assert code == 0 and bool((kept == -1).all()) and torch.equal(pk, pools[0])
