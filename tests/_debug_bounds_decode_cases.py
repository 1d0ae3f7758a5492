"""Small cases of the speculative decoding calls, run once with each build of the
library by test_gpu_debug_bounds_decode.py, in child processes.  Not collected by
pytest (no test_ prefix)."""
import json
import os
import sys

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [HERE, os.path.dirname(HERE)]

import decode_helpers as dh  # noqa: E402
from tree_forked_decision_b200 import flide, inputs  # noqa: E402


def _setup(nodes):
    tree = inputs._tree([(200, [(-1, 2)] + nodes), (33, [(-1, 1), (0, 2)]), (0, [])], 3)
    dt = flide.DeviceTree(*tree.arrays(), max_depth=3)
    idx = flide.TreeIndex(dt.R, dt.N, dt.T, 3)
    flide.tree_build(dt, idx)
    torch.cuda.synchronize()
    return tree, idx


def _calls(tree, idx, d, dtype):
    """Every call once; returns its outputs by name."""
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    T, out = tree.T, {}
    q, k, v = n(T, 8, d).to(dtype).cuda(), n(T, 2, d).to(dtype).cuda(), n(T, 2, d).to(dtype).cuda()
    hist = [[n(int(p), 2, d).to(dtype) for p in tree.past_len] for _ in range(2)]
    pools, table, slots, width = dh.scatter(hist, 64, np.random.default_rng(0), extra=8)
    pk, pv, table, slots = pools[0].cuda(), pools[1].cuda(), table.cuda(), slots.cuda()
    freqs, m = flide.rope_freqs(d)
    out["rope_q"], out["rope_k"] = flide.rope(q, k, idx, freqs, mscale=m)
    out["o"], out["lse"] = flide.draft_attn_paged(q, k, v, idx, 0.1, pk, pv, table, slots, 64, width)
    mass = torch.rand((table.numel() // width, width * 64), generator=g).cuda()
    out["mass"] = flide.history_mass(q, k, out["lse"], idx, 0.1, pk, table, slots, 64, width, mass)
    target, draft = (torch.softmax(n(T, 300), 1).cuda() for _ in range(2))
    tok = torch.randint(0, 300, (T,), generator=g).to(torch.int32).cuda()
    u, un = torch.rand(T, generator=g).cuda(), torch.rand(3, generator=g).cuda()
    out["n"], out["next"], out["path"] = flide.verify_draft(idx, tok, target, u, un, draft=draft)
    torch.cuda.synchronize()
    return out


def run(out_dir):
    res, arrays = {"debug_bounds": int(flide._lib().flide_debug_bounds())}, {}
    chain = [(0, 1), (0, 1), (1, 2), (1, 1)]
    for tag, nodes, d, dtype in (("mma16", [(0, 1)], 64, torch.bfloat16), ("tile32", chain, 128, torch.bfloat16),
                                 ("tile128", chain * 5, 128, torch.bfloat16), ("portable", chain, 96, torch.float32)):
        tree, idx = _setup(nodes)
        for name, x in _calls(tree, idx, d, dtype).items():
            arrays[tag + "_" + name] = x.float().cpu().numpy()
        res["status_" + tag] = idx.status()
    np.savez(os.path.join(out_dir, "arrays.npz"), **arrays)
    with open(os.path.join(out_dir, "result.json"), "w") as f:
        json.dump(res, f)


def run_corrupt(out_dir):
    """Debug build only: an ancestor id, a request's node range and a token's node are overwritten
    with values a little past the tree's counts; the calls report FLIDE_ERR_BOUNDS with the site.
    Each value still lies inside the index's own arrays, so no access leaves device memory even
    without the check."""
    assert flide._lib().flide_debug_bounds() == 1
    res = {}
    for tag, array, at, value in (("ancestor", "anc_node", 1, None), ("token", "token_node", 3, None),
                                  ("range", "req_node", 1, None)):
        tree, idx = _setup([(0, 1), (0, 1), (1, 2), (1, 1)])
        idx.array(array, at + 1)[at] = tree.N + 1
        _calls(tree, idx, 128, torch.bfloat16)
        c = idx.counts()
        res[tag] = [idx.status(), c["CHECK_SITE"], c["CHECK_VALUE"], tree.N + 1]
    with open(os.path.join(out_dir, "corrupt.json"), "w") as f:
        json.dump(res, f)


if __name__ == "__main__":
    torch.cuda.set_device(0)
    (run_corrupt if sys.argv[1] == "corrupt" else run)(sys.argv[2])
