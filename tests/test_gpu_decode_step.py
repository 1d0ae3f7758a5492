"""The speculative decoding operators together: an episode over HistoryStore, against a 64-bit
simulation that keeps each request's history as plain lists; the step in a CUDA graph."""
import math

import numpy as np
import pytest
import torch

from tree_forked_decision_b200 import flide, inputs
from tree_forked_decision_b200.history import HistoryStore

import decode_helpers as dh

pytestmark = pytest.mark.gpu

Hq, Hkv, d, V = 8, 2, 128, 64


def _tree_of(roots, past, rng):
    """Root of the given length and five drafted tokens below it."""
    return inputs._tree([(p, [(-1, n), (0, 1), (0, 1), (1, 2), (1, 1)]) for n, p in zip(roots, past)], 2)


def _turn(x, pos, freqs):
    """Half-layout rotation in 64 bits."""
    n = freqs.shape[0]
    a, b = x.double()[..., :n], x.double()[..., n:]
    ang = torch.outer(torch.as_tensor(pos, dtype=torch.float64), freqs)[:, None]
    return torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1)


@pytest.mark.parametrize("block_rows", [16, 128])
def test_episode(block_rows):
    R, budget, sinks, recent = 3, 24, 2, 8
    rng, g = np.random.default_rng(5), torch.Generator().manual_seed(5)
    width = 128 // block_rows
    store = HistoryStore(n_blocks=R * width + 1, block_rows=block_rows, max_requests=5, max_blocks=width, Hkv=Hkv,
                         d=d)
    slots = [3, 0, 4]
    freqs, m = flide.rope_freqs(d)
    emb = torch.randn(V, (Hq + 2 * Hkv) * d, generator=g)  # token -> its q, k, v
    head = torch.randn(V, Hq * d, generator=g) * 0.4
    past_k = [torch.zeros(0, Hkv, d) for _ in range(R)]     # what the store should hold
    past_v = [torch.zeros(0, Hkv, d) for _ in range(R)]
    mass = [np.zeros(0) for _ in range(R)]
    gone = [0] * R
    roots = [rng.integers(0, V, n).tolist() for n in (30, 25, 3)]
    scale = 1 / math.sqrt(d)
    evicted = 0
    for step in range(6):
        past_len, _ = store.resume_lengths([-1 if store.length(s) == 0 else s for s in slots])
        tree = _tree_of([len(t) for t in roots], [p.shape[0] for p in past_k], rng)
        dt = flide.DeviceTree(*tree.arrays(), max_depth=2)
        idx = flide.TreeIndex(dt.R, dt.N, dt.T, 2)
        flide.tree_build(dt, idx)
        req, pos, sees = dh.layout(tree)
        tokens = np.concatenate([np.concatenate([t, rng.integers(0, V, 5)]) for t in roots])
        x = emb[tokens].to(torch.bfloat16)
        q, k, v = (x[:, a * d:b * d].reshape(-1, b - a, d).contiguous()
                   for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
        qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
        flide.rope(qd, kd, idx, freqs, pos_offset=store.pos_offset(slots), mscale=m, q_out=qd, k_out=kd)
        o, lse = store.draft_attn(qd, kd, vd, idx, scale, slots)
        logits = o.float().reshape(tree.T, -1) @ head.cuda().T / math.sqrt(d)
        target = torch.softmax(logits, 1)
        u, un = torch.rand(tree.T, generator=g), torch.rand(R, generator=g)
        n_acc, nxt, path = flide.verify_draft(idx, torch.from_numpy(tokens.astype(np.int32)).cuda(), target,
                                              u.cuda(), un.cuda())
        store.accumulate_mass(qd, kd, lse, idx, scale, slots)
        store.commit(slots, tree, idx, kd, vd)
        kept = store.evict(slots, budget, sinks=sinks, recent=recent)
        torch.cuda.synchronize()
        assert idx.status() == 0 and int(store.status) == 0

        # the simulation: positions, attention, weights, verification
        off = np.asarray(gone)[req]
        for x16, gpu in ((q, qd), (k, kd)):
            want = _turn(x16, pos + off, freqs.cpu())
            tol = dh.step(torch.bfloat16) * want.abs() + 6e-7 * x16.double().abs().amax(-1, keepdim=True) * 2
            assert bool(((gpu.double().cpu() - want).abs() <= tol).all())
        ow, lw, wv, peak, size = dh.attention(tree, qd.cpu(), kd.cpu(), vd.cpu(), past_k, past_v, scale)
        keys = 128 + tree.T
        err = (o.double().cpu() - ow).abs()
        assert bool((err <= dh.attention_tolerance(ow, wv, peak, size, d, keys, torch.bfloat16, 2.0 ** -8)).all())
        assert bool(((lse.double().cpu() - lw).abs() <= dh.lse_tolerance(lw, size, d, keys)).all())
        n_w, t_w, p_w = dh.verify(tree, tokens, target.cpu().numpy(), None, u.numpy(), un.numpy())
        assert n_acc.tolist() == n_w.tolist() and nxt.tolist() == t_w.tolist() and path.tolist() == p_w.tolist()
        add = dh.mass_of(tree, qd.cpu(), kd.cpu(), past_k, lse.cpu(), scale)
        start = np.concatenate([[0], np.cumsum(tree.seg_len)])
        new_roots = []
        for r in range(R):
            t = slice(start[tree.req_node_ptr[r]], start[tree.req_node_ptr[r] + 1])
            past_k[r] = torch.cat([past_k[r], kd.cpu()[t]])
            past_v[r] = torch.cat([past_v[r], vd.cpu()[t]])
            mass[r] = np.concatenate([mass[r], np.zeros(len(roots[r]))]) + add[r].numpy()
            n = past_k[r].shape[0]
            mine = kept[r].cpu().tolist()
            mine = [i for i in mine if i >= 0]
            # the simulation's weights are 64 bits: rows of the kept set weigh no less than the others
            # within the 32-bit sums' error (1e-5 relative)
            assert len(mine) == min(n, budget) and mine == sorted(mine)
            if n > budget:
                evicted += 1
                lost = sorted(set(range(n)) - set(mine))
                assert set(range(sinks)) <= set(mine) and set(range(n - recent, n)) <= set(mine)
                free = [i for i in mine if sinks <= i < n - recent]
                assert min(mass[r][free]) >= max(mass[r][lost]) * (1 - 1e-5)
                gone[r] += n - budget
            past_k[r], past_v[r], mass[r] = past_k[r][mine], past_v[r][mine], mass[r][mine]
            rows = [int(i) for i in p_w[start[tree.req_node_ptr[r]]:start[tree.req_node_ptr[r + 1]]] if i >= 0]
            new_roots.append([int(tokens[i]) for i in rows] + [int(t_w[r])])
        # the store holds the simulation's history
        table = store.table.cpu().view(5, width)
        for r, s in enumerate(slots):
            n = store.length(s)
            at = table[s][torch.arange(n) // block_rows].long() * block_rows + torch.arange(n) % block_rows
            assert torch.equal(store.pool_k.cpu()[at], past_k[r]) and torch.equal(store.pool_v.cpu()[at], past_v[r])
            assert np.allclose(store.mass.cpu()[s, :n].numpy(), mass[r], rtol=1e-5)
            if len([i for i in kept[r].tolist() if i >= 0]) == budget:  # rows to come start without weight
                assert not bool(store.mass[s, budget:].any())
        assert store.pos_offset(slots).tolist() == gone
        assert store.free_blocks() == R * width + 1 - sum(-(-store.length(s) // block_rows) for s in slots)
        roots = new_roots
        if step == 3:  # an episode ends: its slot starts over
            store.release(slots[1])
            past_k[1], past_v[1], mass[1], gone[1] = past_k[1][:0], past_v[1][:0], mass[1][:0], 0
            assert store.pos_offset(slots).tolist() == gone
    assert evicted > 3


def test_step_in_a_graph():
    """rope, attention, verification and weights captured once and replayed on other values give the
    eager calls' bits; a second graph over the same workspace, replayed after it, too."""
    rng = np.random.default_rng(1)
    tree = inputs._tree([(500, [(-1, 2), (0, 1), (0, 1), (1, 1)]), (77, [(-1, 1), (0, 2)])], 2)
    dt = flide.DeviceTree(*tree.arrays(), max_depth=2)
    idx = flide.TreeIndex(dt.R, dt.N, dt.T, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    hist = [[torch.randn(p, Hkv, d).bfloat16() for p in (500, 77)] for _ in range(2)]
    pools, table, slots, width = dh.scatter(hist, 64, rng, extra=8)
    pk, pv, table, slots = pools[0].cuda(), pools[1].cuda(), table.cuda(), slots.cuda()
    freqs, m = flide.rope_freqs(d)
    T = tree.T
    q, k, v = n(T, Hq, d).bfloat16(), n(T, Hkv, d).bfloat16(), n(T, Hkv, d).bfloat16()
    target, u, un = torch.softmax(n(T, V), 1), torch.rand(T, device="cuda"), torch.rand(2, device="cuda")
    tok = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    mass = torch.rand((table.numel() // width, width * 64), device="cuda")
    ws = flide.draft_attn_workspace(idx, Hq, Hkv, d)
    bufs = [torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty(T, Hq, device="cuda"),
            torch.empty_like(mass)]
    outs = [torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"),
            torch.empty(T, dtype=torch.int32, device="cuda")]

    def step(scale=0.09):
        flide.tree_build(dt, idx)
        flide.rope(q, k, idx, freqs, mscale=m, q_out=bufs[0], k_out=bufs[1])
        flide.draft_attn_paged(bufs[0], bufs[1], v, idx, scale, pk, pv, table, slots, 64, width, out=bufs[2],
                               lse=bufs[3], workspace=ws)
        flide.verify_draft(idx, tok, target, u, un, n_accept=outs[0], next_token=outs[1], path=outs[2])
        flide.history_mass(bufs[0], bufs[1], bufs[3], idx, scale, pk, table, slots, 64, width, mass,
                           mass_out=bufs[4])

    step()
    torch.cuda.synchronize()
    graphs = []
    for scale in (0.09, 0.05):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(scale)
        graphs.append((graph, scale))
    for i in range(3):
        q.copy_(n(T, Hq, d))
        pk.copy_(n(*pk.shape))
        target.copy_(torch.softmax(2 * n(T, V), 1))
        u.uniform_()
        for graph, scale in graphs:
            bufs[4].copy_(mass)
            graph.replay()
            torch.cuda.synchronize()
            got = [x.clone() for x in bufs + outs]
            bufs[4].copy_(mass)
            step(scale)
            torch.cuda.synchronize()
            assert idx.status() == 0
            for a, b in zip(got, bufs + outs):
                assert torch.equal(a, b)
