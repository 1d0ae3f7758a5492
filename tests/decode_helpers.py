"""Plain 64-bit forms of the speculative decoding operators, for their tests."""
import math

import numpy as np
import torch


def layout(tree):
    """Per stream token: request, isolated position, visible stream rows (its path)."""
    rp, parent, seg, past = tree.arrays()
    start = np.concatenate([[0], np.cumsum(seg)]).astype(int)
    req, pos, sees = [], [], []
    for r in range(len(rp) - 1):
        chain = {}
        for n in range(rp[r], rp[r + 1]):
            above = [] if parent[n] < 0 else chain[rp[r] + parent[n]]
            rows = list(range(start[n], start[n + 1]))
            chain[n] = above + rows
            for i, t in enumerate(rows):
                req.append(r)
                sees.append(above + rows[:i + 1])
                pos.append(int(past[r]) + len(above) + i)
    return np.asarray(req, int), np.asarray(pos, int), sees


def step(t):
    """Largest relative error of a rounding to t's type."""
    return {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[t]


def attention(tree, q, k, v, pk, pv, scale):
    """(o, lse, sum of w |v|, largest w times the sum of |v|, largest sum of |q k| * scale) per token
    and head, in 64 bits; pk, pv: a list of each request's history rows."""
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    q, k, v = (x.double() for x in (q, k, v))
    req, _, sees = layout(tree)
    o, lse = torch.zeros(T, Hq, d, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    wv, peak, size = torch.zeros_like(o), torch.zeros_like(o), 0.0
    for t in range(len(req)):
        kk = torch.cat([pk[req[t]].double(), k[sees[t]]]).repeat_interleave(G, 1)
        vv = torch.cat([pv[req[t]].double(), v[sees[t]]]).repeat_interleave(G, 1)
        s = torch.einsum("hd,nhd->hn", q[t], kk) * scale
        size = max(size, float((torch.einsum("hd,nhd->hn", q[t].abs(), kk.abs()) * scale).max()))
        lse[t] = torch.logsumexp(s, 1)
        w = torch.softmax(s, 1)
        o[t] = torch.einsum("hn,nhd->hd", w, vv)
        wv[t] = torch.einsum("hn,nhd->hd", w, vv.abs())
        peak[t] = w.amax(1, keepdim=True) * vv.abs().sum(0)
    return o, lse, wv, peak, size


def attention_tolerance(o, wv, peak, size, d, keys, out_type, weight_step, weight_least=0.0):
    """Elementwise bound: the output's rounding, the rounded weights (off by weight_step of
    themselves, or weight_least of the row's largest), and 32-bit sums.
    A score is d products summed in 32 bits, off by at most (d + 4) 2^-24 of the sum of
    their sizes; that shifts its weight and the total by the same factor (hence 2 x).
    exp2 and its argument add 2^-20; keys 32-bit additions (keys + 8) 2^-24."""
    ds = (d + 4) * 2.0 ** -24 * size
    return step(out_type) * o.abs() + (weight_step + 2 * ds + 2.0 ** -20 + 2 * (keys + 8) * 2.0 ** -24) * wv \
        + weight_least * peak + 1e-12


def lse_tolerance(lse, size, d, keys):
    return (d + 4) * 2.0 ** -24 * size + (keys + 8) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * lse.abs()


def mass_of(tree, q, k, pk, lse, scale):
    """Per request: weight that its root tokens gave its history rows and its root rows."""
    rp, _, seg, _ = tree.arrays()
    start = np.concatenate([[0], np.cumsum(seg)]).astype(int)
    G = q.shape[1] // k.shape[1]
    got = []
    for r in range(tree.R):
        if rp[r + 1] == rp[r] or seg[rp[r]] == 0:
            got.append(None)
            continue
        t = torch.arange(start[rp[r]], start[rp[r] + 1])
        kk = torch.cat([pk[r].double(), k[t].double()]).repeat_interleave(G, 1)
        w = torch.exp(torch.einsum("thd,nhd->thn", q[t].double(), kk) * scale - lse[t].double()[..., None])
        hide = torch.arange(len(t))[:, None] < torch.arange(len(t))[None]
        w[:, :, pk[r].shape[0]:] *= (~hide).double()[:, None]
        got.append(w.sum((0, 1)))
    return got


def verify(tree, tokens, target, draft, u, u_next):
    """The residual rejection rule as it is stated: the residual itself is kept and
    normalised after every rejection."""
    rp, parent, seg, _ = tree.arrays()
    start = np.concatenate([[0], np.cumsum(seg)]).astype(int)
    clean = lambda x: np.where(np.asarray(x, np.float64) > 0, np.asarray(x, np.float64), 0.0)  # noqa: E731
    T = int(start[-1])
    path, count, nxt = np.full(T, -1, int), [], []
    for r in range(tree.R):
        nodes = range(rp[r], rp[r + 1])
        if len(nodes) == 0 or seg[rp[r]] == 0:
            count.append(0)
            nxt.append(-1)
            continue
        node, at, taken = rp[r], start[rp[r] + 1] - 1, []
        while True:
            p = clean(target[at])
            res, total, seen = p.copy(), 1.0, set()
            kids = [(node, at + 1)] if at + 1 < start[node + 1] else \
                [(m, start[m]) for m in nodes if parent[m] >= 0 and rp[r] + parent[m] == node]
            down = None
            for m, row in kids:
                x = int(tokens[row])
                if not 0 <= x < len(p):
                    continue
                if draft is not None:
                    q = clean(draft[at])
                    if float(u[row]) * q[x] < res[x]:
                        down = (m, row)
                    else:
                        res = np.maximum(res - q, 0.0)
                        res = res / res.sum() if res.sum() > 0 else res
                elif x not in seen:
                    if float(u[row]) * total < res[x]:
                        down = (m, row)
                    else:
                        total -= res[x]
                        res[x] = 0.0
                        seen.add(x)
                if down:
                    break
            if down is None:
                break
            node, at = down
            taken.append(at)
        if not res.sum() > 0:
            res = p
        cum = np.cumsum(res)
        pick = int(np.searchsorted(cum, float(u_next[r]) * cum[-1], side="right"))
        nxt.append(min(pick, int(np.flatnonzero(res > 0)[-1])) if cum[-1] > 0 else -1)
        path[start[rp[r]]:start[rp[r]] + len(taken)] = taken
        count.append(len(taken))
    return np.asarray(count), np.asarray(nxt), path


def keep_rows(mass, n, budget, sinks, recent):
    """Ascending rows that an eviction keeps (a NaN is below every number, -inf included)."""
    if n <= budget:
        return list(range(n))
    fixed = set(range(sinks)) | set(range(n - recent, n))
    key = [(1, 0.0) if math.isnan(m) else (0, -float(m)) for m in mass[:n]]
    rest = sorted((i for i in range(n) if i not in fixed), key=lambda i: (key[i], i))
    return sorted(fixed | set(rest[:budget - len(fixed)]))


def scatter(rows, block_rows, rng, spare_blocks=2, spare_slots=1, extra=0, fill=None):
    """Pools (one per list in `rows`: each request's rows), table, slots, width: the rows in
    random blocks, room for `extra` more each; other pool rows hold `fill` (default 0)."""
    R = len(rows[0])
    need = [-(-(x.shape[0] + extra) // block_rows) for x in rows[0]]
    n_blocks, width = max(sum(need) + spare_blocks, 1), max(need + [1])
    slots = rng.permutation(R + spare_slots)[:R].astype(np.int32)
    free = list(rng.permutation(n_blocks))
    table = np.full((R + spare_slots, width), -1, np.int32)
    pools = []
    for x in rows:
        pool = torch.zeros((n_blocks * block_rows,) + tuple(x[0].shape[1:]), dtype=torch.float32)
        pool += 0.0 if fill is None else fill
        pools.append(pool.to(x[0].dtype))
    for r in range(R):
        for b in range(need[r]):
            blk = int(free.pop())
            table[slots[r], b] = blk
            for pool, x in zip(pools, rows):
                part = x[r][b * block_rows:(b + 1) * block_rows]
                pool[blk * block_rows:blk * block_rows + part.shape[0]] = part
    return pools, torch.from_numpy(table.ravel().copy()), torch.from_numpy(slots), width
