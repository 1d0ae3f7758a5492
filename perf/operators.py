"""Cases that time the operators of one speculative decoding step over a paged history.

A serving step continues each request's history with a small tree: a root (the
tokens committed since the last step) and drafted tokens below it.  The
operators, in the order the step uses them: rotary positions of the tree
(``rope``), attention of the tree over the history (``draft``), verification of
the drafted tokens (``verify``), the attention weight that the history's rows
gathered (``mass``) and the eviction of the rows with the least (``evict``).

``run`` computes them in elementary torch operations when ``own`` is false and
through the package's entry points when it is true; ``exact`` states them in 64
bits.  Shapes follow from the case alone, values from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.uint8}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}


# ---- cases --------------------------------------------------------------------------------

def listed():
    return [
        # the step of a single tree: a few tokens, where only latency counts
        dict(name="rope_step", op="rope", shape=1, R=8, root=1, nodes=4, blen=1, past=8192, ragged=True,
             Hq=16, Hkv=4, d=128, rot=128, inter=False, scaling="none", dtype="bf16"),
        # a batch of prompts with their options: bandwidth; the GDN fan-out's tree with the large fan-out's heads
        dict(name="rope_prefill", op="rope", shape=2, R=8, root=4096, nodes=64, blen=16, past=0, ragged=False,
             Hq=32, Hkv=8, d=128, rot=128, inter=True, scaling="yarn", dtype="bf16"),
        # one user, a short history, the smallest tree
        dict(name="draft_one", op="draft", shape=3, R=1, root=1, nodes=4, blen=1, past=2048, ragged=False,
             Hq=16, Hkv=4, d=128, dtype="bf16", block=128),
        # a ragged batch, small trees, small pages
        dict(name="draft_batch", op="draft", shape=4, R=16, root=2, nodes=9, blen=2, past=8192, ragged=True,
             Hq=32, Hkv=8, d=128, dtype="bf16", block=16),
        # long histories and wide trees: bandwidth and tensor cores both near their limits
        dict(name="draft_wide", op="draft", shape=5, R=8, root=4, nodes=60, blen=1, past=32768, ragged=False,
             Hq=32, Hkv=8, d=128, dtype="bf16", block=128),
        # an 8-bit history, packed, odd lengths
        dict(name="draft_e4m3", op="draft", shape=6, R=16, root=1, nodes=7, blen=1, past=16391, ragged=True,
             Hq=32, Hkv=8, d=128, dtype="e4m3", block=0),
        # weights gathered after a step: one user, and a batch of long histories
        dict(name="mass_small", op="mass", shape=7, R=2, root=2, nodes=0, blen=1, past=1500, ragged=True,
             Hq=16, Hkv=4, d=128, dtype="bf16", block=128),
        dict(name="mass_large", op="mass", shape=8, R=16, root=4, nodes=0, blen=1, past=16384, ragged=True,
             Hq=32, Hkv=8, d=128, dtype="bf16", block=128),
        # a few rows over a small budget, and a batch cut to half of a long history
        dict(name="evict_small", op="evict", shape=9, R=2, past=2304, ragged=True, budget=2048, sinks=4,
             recent=64, Hkv=4, d=128, dtype="bf16", block=128),
        dict(name="evict_large", op="evict", shape=10, R=16, past=16384, ragged=False, budget=8192, sinks=4,
             recent=512, Hkv=8, d=128, dtype="bf16", block=128),
        # greedily drafted tokens of one user under the decision head's vocabulary
        dict(name="verify_point", op="verify", shape=11, R=1, root=1, nodes=6, blen=1, V=8192, sampled=False,
             dtype="f32"),
        # a batch of sampled trees under a large vocabulary
        dict(name="verify_sampled", op="verify", shape=12, R=64, root=1, nodes=12, blen=2, V=131072, sampled=True,
             dtype="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "draft", "draft", "mass", "evict", "verify"])
    c = dict(op=op, shape=rng.randrange(1 << 30), R=_log(rng, 1, 16))
    heads = rng.choice([(8, 8), (16, 4), (32, 8), (12, 3), (16, 2), (5, 5)])
    if op == "rope":
        d = rng.choice([64, 80, 128])
        c.update(root=_log(rng, 1, 1024), nodes=rng.randrange(0, 33), blen=rng.choice([1, 3, 16]),
                 past=_log(rng, 1, 1 << 20), ragged=rng.random() < 0.6, Hq=heads[0], Hkv=heads[1], d=d,
                 rot=rng.choice([d, d // 2, 32]), inter=rng.random() < 0.5,
                 scaling=rng.choice(["none", "linear", "ntk", "yarn"]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    elif op in ("draft", "mass"):
        dtype = rng.choice(["bf16", "bf16", "e4m3", "f32"])
        c.update(root=rng.choice([1, 1, 2, 5, 9]), nodes=rng.choice([0, 3, 8, 21, 50]) if op == "draft" else 0,
                 blen=rng.choice([1, 1, 3]), past=_log(rng, 1, 16384), ragged=rng.random() < 0.6, Hq=heads[0],
                 Hkv=heads[1], d=128 if dtype == "e4m3" else rng.choice([64, 128]), dtype=dtype,
                 block=rng.choice([16, 48, 128, 256] + ([0] if op == "draft" else [])))
        if c["nodes"] > 21:
            c["blen"] = 1
        if dtype == "f32":
            c["past"] = min(c["past"], 4096)
    elif op == "evict":
        past = _log(rng, 64, 16384)
        budget = max(8, int(past * rng.uniform(0.3, 1.1)))
        c.update(past=past, ragged=rng.random() < 0.6, budget=budget, sinks=rng.randrange(0, 5),
                 recent=rng.randrange(0, budget // 2), Hkv=heads[1], d=rng.choice([64, 128]),
                 dtype=rng.choice(["bf16", "bf16", "e4m3", "f32"]), block=rng.choice([16, 48, 128]))
    else:
        c.update(root=rng.choice([1, 1, 3]), nodes=rng.randrange(0, 25), blen=rng.choice([1, 1, 2]),
                 V=_log(rng, 257, 131072), sampled=rng.random() < 0.6, dtype=rng.choice(["f32", "f32", "bf16"]))
    return c


# ---- shapes, from the case alone -----------------------------------------------------------

def _lengths(case):
    rng = random.Random(case["shape"])
    n = case["past"]
    return [n if not case["ragged"] or r == 0 else rng.randint(n // 16, n) for r in range(case["R"])]


def _tree(case, past):
    """(req_node_ptr, parent, seg_len, past_len) of the batch and its depth: a root of `root`
    tokens and `nodes` branch nodes of up to `blen` tokens, hung below random earlier nodes."""
    rng = random.Random(case["shape"] + 1)
    rp, parent, seg, deepest = [0], [], [], 0
    fan = case["nodes"] * case["blen"] >= 512  # a prompt's options: equal leaves
    for _ in range(case["R"]):
        parent.append(-1)
        seg.append(case["root"])
        depth = [0]
        for i in range(case["nodes"]):
            pa = 0 if fan else rng.choice([j for j in range(max(0, i - 6), i + 1) if depth[j] < 6] or [0])
            parent.append(pa)
            seg.append(case["blen"] if fan else rng.randint(1, case["blen"]))
            depth.append(depth[pa] + 1)
        deepest = max(deepest, max(depth))
        rp.append(len(parent))
    i32 = lambda a: np.asarray(a, np.int32)  # noqa: E731
    return (i32(rp), i32(parent), i32(seg), i32(past)), deepest


def _layout(arrays):
    """Per stream token: request, position in its isolated sequence, the row before it on its path
    (-1 for a request's first token), last-token row of each root; [T, T] visibility."""
    rp, parent, seg, past = arrays
    start = np.concatenate([[0], np.cumsum(seg)])
    T = int(start[-1])
    req, pos, prev = np.zeros(T, np.int64), np.zeros(T, np.int64), np.full(T, -1, np.int64)
    tail = np.zeros(len(rp) - 1, np.int64)
    for r in range(len(rp) - 1):
        for n in range(rp[r], rp[r + 1]):
            s, e = start[n], start[n + 1]
            last = -1 if parent[n] < 0 else start[rp[r] + parent[n] + 1] - 1
            req[s:e] = r
            pos[s:e] = np.arange(e - s) + (past[r] if last < 0 else pos[last] + 1)
            prev[s:e] = np.concatenate([[last], np.arange(s, e - 1)])
        tail[r] = start[rp[r] + 1] - 1
    return req, pos, prev, tail, T


def _visible(prev, T):
    see = np.zeros((T, T), bool)
    for t in range(T):
        if prev[t] >= 0:
            see[t] = see[prev[t]]
        see[t, t] = True
    return see


def work(case):
    e, op = SIZE[case["dtype"]], case["op"]
    R = case["R"]
    if op == "rope":
        T = _layout(_tree(case, [0] * R)[0])[4]
        n = T * (case["Hq"] + case["Hkv"])
        return dict(bytes=2 * n * case["d"] * e, flops=3 * n * case["rot"])
    if op == "verify":
        return dict(bytes=R * case["V"] * e * (2 if case["sampled"] else 1),
                    flops=R * case["V"] * (3 if case["sampled"] else 1))
    past = sum(_lengths(case))
    if op == "evict":
        kept = sum(min(n, case["budget"]) for n in _lengths(case))
        return dict(bytes=kept * 4 * case["Hkv"] * case["d"] * e + 4 * past + 8 * kept, flops=past)
    arrays, _ = _tree(case, _lengths(case))
    T = int(arrays[2].sum())
    n = T // R if op == "draft" else case["root"]  # tokens that look at the history (mean per request)
    stream = T * case["d"] * (2 * case["Hq"] + 2 * case["Hkv"]) * e
    if op == "draft":
        return dict(bytes=2 * past * case["Hkv"] * case["d"] * e + stream, flops=4 * case["d"] * case["Hq"] * n * past)
    own_rows = T * (case["d"] * (case["Hq"] + case["Hkv"]) * e + 4 * case["Hq"])
    return dict(bytes=past * case["Hkv"] * case["d"] * e + 8 * past + own_rows, flops=2 * case["d"] * case["Hq"] * n * past)


# ---- inputs --------------------------------------------------------------------------------

def _dev(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV)


def _handle(s, arrays, depth):
    """The tree index that a step keeps for all its layers."""
    if own:
        from tree_forked_decision_b200 import flide
        tree = flide.DeviceTree(*arrays, max_depth=depth)
        s["index"] = flide.TreeIndex(tree.R, tree.N, tree.T, tree.max_depth)
        flide.tree_build(tree, s["index"])


def _codes(x, amax):
    """e4m3 codes as bytes, and the factor that gives their values."""
    return (x * (448.0 / amax)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), amax / 448.0


def _pages(case, lens, extra):
    """A shuffled block table for slots of these lengths (+ extra rows), slots in another order than requests."""
    rng = np.random.default_rng(case["shape"] + 2)
    bl, R = case["block"], len(lens)
    need = [-(-(n + extra) // bl) for n in lens]
    width, n_slots = max(max(need), 1), R + 1
    slots = rng.permutation(n_slots)[:R].astype(np.int32)
    n_blocks = max(sum(need), 1)
    ids, table, at = rng.permutation(n_blocks).astype(np.int32), np.full((n_slots, width), -1, np.int32), 0
    for r, m in enumerate(need):
        table[slots[r], :m] = ids[at:at + m]
        at += m
    return table, slots, n_blocks, width


def _rows_of(table, slots, lens, bl):
    """Pool rows of the requests' histories, padded: [R, longest] (padding: row 0)."""
    i = np.arange(max(max(lens), 1))
    rows = np.maximum(table[slots][:, np.minimum(i // bl, table.shape[1] - 1)], 0).astype(np.int64) * bl + i % bl
    return np.where(i[None] < np.asarray(lens)[:, None], rows, 0)


def _qkv(case, T, P, g):
    """Queries, the step's keys and values and P history rows; a shared direction makes some rows draw
    more weight than others."""
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    n = lambda *sh: torch.randn(sh, generator=g, device=DEV)  # noqa: E731
    way = n(Hkv, d)
    way = way / way.norm(dim=-1, keepdim=True)
    q = n(T, Hq, d) + 3.0 * way.repeat_interleave(Hq // Hkv, 0)
    k = n(T, Hkv, d) + 2.0 * n(T, Hkv, 1) * way
    pk = n(P, Hkv, d)
    pk += 4.0 * n(P, 1, 1) * way
    v, pv = n(T, Hkv, d), n(P, Hkv, d)
    if case["dtype"] != "e4m3":
        return [x.to(TYPES[case["dtype"]]) for x in (q, k, v, pk, pv)] + [None]
    (q, sq), (k, sk), (v, sv) = _codes(q, 10.0), _codes(k, 18.0), _codes(v, 6.0)
    pk, pv = _codes(pk, 18.0)[0], _codes(pv, 6.0)[0]
    return [q, k, v, pk, pv, torch.tensor([sq, sk, sv], device=DEV)]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, s = case["op"], {"case": case}
    if op == "evict":
        return _prepare_evict(case, s, g)
    past = [0] * case["R"] if op == "verify" else _lengths(case)
    arrays, depth = _tree(case, past)
    req, pos, prev, tail, T = _layout(arrays)
    _handle(s, arrays, depth)
    if op == "rope":
        # rows evicted so far shift each request's positions
        off = np.random.default_rng(seed).integers(0, 5000, case["R"]).astype(np.int32)
        s.update(pos=_dev(pos), req=_dev(req), offset=_dev(off))
        s["freqs"], s["mscale"] = _freqs(case)
        for name, H in (("q", case["Hq"]), ("k", case["Hkv"])):
            s[name] = torch.randn((T, H, case["d"]), generator=g, device=DEV).to(TYPES[case["dtype"]])
            s[name + "_out"] = torch.empty_like(s[name])
        return s
    if op == "verify":
        return _prepare_verify(case, s, g, prev, tail, T)
    s["scale"] = 1.0 / math.sqrt(case["d"])
    if case["block"]:
        table, slots, n_blocks, width = _pages(case, past, case["root"])
        s["q"], s["k"], s["v"], s["pk"], s["pv"], s["descale"] = _qkv(case, T, n_blocks * case["block"], g)
        s.update(table=_dev(table.ravel()), slots=_dev(slots), width=width)
        rows = _rows_of(table, slots, past, case["block"])
    else:
        s["q"], s["k"], s["v"], s["pk"], s["pv"], s["descale"] = _qkv(case, T, sum(past), g)
        first = np.concatenate([[0], np.cumsum(past)[:-1]])
        i = np.arange(max(max(past), 1))
        rows = np.where(i[None] < np.asarray(past)[:, None], first[:, None] + i, 0)
    # the plain form's plan: rows of each history, each request's stream rows, who sees whom
    most = int(np.bincount(req, minlength=case["R"]).max())
    toks = np.full((case["R"], most), -1, np.int64)
    for r in range(case["R"]):
        t = np.flatnonzero(req == r)
        toks[r, :len(t)] = t
    see = np.take_along_axis(_visible(prev, T)[np.maximum(toks, 0)], np.maximum(toks, 0)[:, None, :], 2) \
        & (toks >= 0)[:, None, :] & (toks >= 0)[:, :, None]
    s.update(rows=_dev(rows), past=_dev(np.asarray(past, np.int64)), toks=_dev(toks), see=_dev(see), lens=past)
    if op == "mass":
        s["cap"] = s["width"] * case["block"]
        s["mass"] = torch.rand((case["R"] + 1, s["cap"]), generator=g, device=DEV)
        s["mass_out"] = s["mass"].clone()
        s["roots"] = _dev(np.stack([np.arange(t - case["root"] + 1, t + 1) for t in tail]))
        s["lse"] = _plain_draft(s)[1]
    else:
        s["out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16 if case["dtype"] == "e4m3" else s["q"].dtype, device=DEV)
        s["lse"] = torch.empty((T, case["Hq"]), device=DEV)
        if own:
            from tree_forked_decision_b200 import flide
            s["workspace"] = flide.draft_attn_workspace(s["index"], case["Hq"], case["Hkv"], case["d"])
    return s


def _freqs(case):
    """Radians a position for each rotated pair, as a table of 64-bit floats, and the factor of long contexts."""
    n, base, f = case["rot"] // 2, 10000.0, 8.0
    if case["scaling"] == "ntk":
        base *= f ** (case["rot"] / (case["rot"] - 2)) if case["rot"] > 2 else 1.0
    w = base ** (-2.0 * np.arange(n) / case["rot"])
    if case["scaling"] == "linear":
        w = w / f
    if case["scaling"] == "yarn":
        turns = 4096 * w / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return _dev(w * (keep + (1 - keep) / f)), 0.1 * math.log(f) + 1.0
    return _dev(w), 1.0


def _prepare_evict(case, s, g):
    lens = _lengths(case)
    table, slots, n_blocks, width = _pages(case, lens, 0)
    rows = n_blocks * case["block"]
    kind = TYPES[case["dtype"]]
    for name in ("pk", "pv"):
        x = torch.randn((rows, case["Hkv"], case["d"]), generator=g, device=DEV)
        s[name] = _codes(x, 6.0)[0] if case["dtype"] == "e4m3" else x.to(kind)
    # attention weight gathers on few rows; equal values occur (rows that were never looked at)
    cap = width * case["block"]
    m = torch.exp(2.0 * torch.randn((len(lens) + 1, cap), generator=g, device=DEV))
    s["mass"] = torch.where(torch.rand(m.shape, generator=g, device=DEV) < 0.1, 0.0, m)
    # the kept rows go to blocks of their own (the old ones may be shared with other forks of the history)
    kept = [min(n, case["budget"]) for n in lens]
    need = [-(-n // case["block"]) for n in kept]
    to, at = np.full((len(lens) + 1, width), -1, np.int32), 0
    for r, m in enumerate(need):
        to[slots[r], :m] = np.arange(at, at + m)
        at += m
    s["dst_k"] = torch.zeros((at * case["block"],) + s["pk"].shape[1:], dtype=kind, device=DEV)
    s["dst_v"] = torch.zeros_like(s["dst_k"])
    s["mass_out"] = torch.zeros_like(s["mass"])
    s["kept"] = torch.full((len(lens), case["budget"]), -1, dtype=torch.int32, device=DEV)
    hist = np.zeros(len(lens) + 1, np.int32)
    hist[slots] = lens
    s.update(table=_dev(table.ravel()), slots=_dev(slots), width=width, cap=cap, hist=_dev(hist),
             to=_dev(to.ravel()), lens=lens, status=torch.zeros(1, dtype=torch.int32, device=DEV))
    return s


def _prepare_verify(case, s, g, prev, tail, T):
    V, kind = case["V"], TYPES[case["dtype"]]
    logits = 3.0 * torch.randn((T, V), generator=g, device=DEV)
    near = logits + 0.5 * torch.randn((T, V), generator=g, device=DEV)  # the draft model: close to the target
    kids = [np.flatnonzero(prev == t) for t in range(T)]
    most = max([len(k) for k in kids] + [1])
    table = np.full((T, most), -1, np.int64)
    rank = np.zeros(T, np.int64)
    for t, k in enumerate(kids):
        table[t, :len(k)] = k
        rank[k] = np.arange(len(k))
    before = _dev(np.maximum(prev, 0))
    s["target"] = torch.softmax(logits, -1).to(kind)
    near = torch.softmax(near, -1)
    if case["sampled"]:
        s["draft"] = near.to(kind)
        s["tokens"] = torch.cat([torch.multinomial(near[before[i:i + 64]], 1, generator=g)[:, 0]
                                 for i in range(0, T, 64)]).to(torch.int32)
    else:
        s["draft"] = None
        top = near.topk(most, dim=-1).indices
        s["tokens"] = top[before, _dev(rank)].to(torch.int32)
    s["u"] = torch.rand(T, generator=g, device=DEV)
    s["u_next"] = torch.rand(case["R"], generator=g, device=DEV)
    down = np.zeros(T, np.int64)
    for t in range(T):
        down[t] = down[prev[t]] + 1 if prev[t] >= 0 else 0
    s.update(kids=_dev(table), tail=_dev(tail), first=_dev(tail - case["root"] + 1),
             levels=int(down.max()) - case["root"] + 2)
    s["n_accept"] = torch.empty(case["R"], dtype=torch.int32, device=DEV)
    s["next_token"] = torch.empty(case["R"], dtype=torch.int32, device=DEV)
    s["path"] = torch.empty(T, dtype=torch.int32, device=DEV)
    return s


# ---- one pass ------------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "draft": _plain_draft, "mass": _plain_mass, "evict": _plain_evict,
                "verify": _plain_verify}[op](s)
    from tree_forked_decision_b200 import flide
    case = s["case"]
    if op == "rope":
        return flide.rope(s["q"], s["k"], s["index"], s["freqs"], pos_offset=s["offset"], mscale=s["mscale"],
                          interleaved=case["inter"], q_out=s["q_out"], k_out=s["k_out"])
    if op == "draft" and case["block"]:
        return flide.draft_attn_paged(s["q"], s["k"], s["v"], s["index"], s["scale"], s["pk"], s["pv"], s["table"],
                                      s["slots"], case["block"], s["width"], descale=s["descale"], out=s["out"],
                                      lse=s["lse"], workspace=s["workspace"])
    if op == "draft":
        return flide.draft_attn(s["q"], s["k"], s["v"], s["index"], s["scale"], past_k=s["pk"], past_v=s["pv"],
                                descale=s["descale"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    if op == "mass":
        return flide.history_mass(s["q"], s["k"], s["lse"], s["index"], s["scale"], s["pk"], s["table"], s["slots"],
                                  case["block"], s["width"], s["mass"], mass_out=s["mass_out"], descale=s["descale"])
    if op == "evict":
        kept = flide.history_evict(s["slots"], s["hist"], s["table"], case["block"], s["width"], s["pk"], s["pv"],
                                   s["mass"], case["budget"], s["status"], sinks=case["sinks"], recent=case["recent"],
                                   dst_k=s["dst_k"], dst_v=s["dst_v"], dst_table=s["to"], mass_out=s["mass_out"],
                                   kept=s["kept"])
        return kept, _value(s, s["dst_k"]), _value(s, s["dst_v"]), s["mass_out"]
    return flide.verify_draft(s["index"], s["tokens"], s["target"], s["u"], s["u_next"], draft=s["draft"],
                              n_accept=s["n_accept"], next_token=s["next_token"], path=s["path"])


def _value(s, x):
    """8-bit rows as the values they stand for (their type's own reading)."""
    return x.view(torch.float8_e4m3fn) if s["case"]["dtype"] == "e4m3" else x


def _plain_rope(s):
    n = s["case"]["rot"] // 2
    angle = (s["pos"] + s["offset"][s["req"]]).double()[:, None] * s["freqs"]
    cos, sin = (s["mscale"] * f(angle).float()[:, None] for f in (torch.cos, torch.sin))
    got = []
    for x in (s["q"], s["k"]):
        f = x.float()
        if s["case"]["inter"]:
            a, b = f[..., 0:2 * n:2], f[..., 1:2 * n:2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = f[..., :n], f[..., n:2 * n]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        got.append(torch.cat([y, f[..., 2 * n:]], -1).to(x.dtype))
    return got


def _number(s, x, which):
    """Stored rows as 32-bit values."""
    return x.view(torch.float8_e4m3fn).float() * s["descale"][which] if s["descale"] is not None else x.float()


def _plain_draft(s):
    case, toks = s["case"], s["toks"].clamp(min=0)
    G = case["Hq"] // case["Hkv"]
    R, n = toks.shape
    q = _number(s, s["q"][toks], 0).view(R, n, case["Hkv"], G, case["d"])
    k = torch.cat([_number(s, s["pk"][s["rows"]], 1) if len(s["pk"]) else q.new_zeros(R, 0, case["Hkv"], case["d"]),
                   _number(s, s["k"][toks], 1)], 1)
    v = torch.cat([_number(s, s["pv"][s["rows"]], 2) if len(s["pv"]) else q.new_zeros(R, 0, case["Hkv"], case["d"]),
                   _number(s, s["v"][toks], 2)], 1)
    L = k.shape[1] - n
    seen = torch.cat([(torch.arange(L, device=q.device) < s["past"][:, None])[:, None].expand(R, n, L), s["see"]], 2)
    x = torch.einsum("rnhgd,rlhd->rhgnl", q, k) * s["scale"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    w = torch.exp(x - top)
    total = w.sum(-1, keepdim=True)
    o = torch.einsum("rhgnl,rlhd->rnhgd", w / total.clamp(min=1e-38), v).reshape(R, n, case["Hq"], case["d"])
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(R, n, case["Hq"])
    real = s["toks"] >= 0
    kind = torch.bfloat16 if case["dtype"] == "e4m3" else s["q"].dtype
    out = torch.empty(s["q"].shape, dtype=kind, device=q.device)
    out[toks[real]] = o[real].to(kind)
    back = torch.empty(s["q"].shape[:2], device=q.device)
    back[toks[real]] = lse[real]
    return out, back


def _plain_mass(s):
    case, roots = s["case"], s["roots"]
    G = case["Hq"] // case["Hkv"]
    R, n = roots.shape
    q = _number(s, s["q"][roots], 0).view(R, n, case["Hkv"], G, case["d"])
    k = torch.cat([_number(s, s["pk"][s["rows"]], 1), _number(s, s["k"][roots], 1)], 1)
    L = k.shape[1] - n
    seen = torch.cat([(torch.arange(L, device=q.device) < s["past"][:, None])[:, None].expand(R, n, L),
                      torch.ones(n, n, dtype=torch.bool, device=q.device).tril()[None].expand(R, n, n)], 2)
    x = torch.einsum("rnhgd,rlhd->rnlhg", q, k) * s["scale"] - s["lse"][roots].view(R, n, 1, case["Hkv"], G)
    w = torch.where(seen[..., None, None], torch.exp(x), 0.0).sum((1, 3, 4))
    to = s["mass_out"]
    slot = s["slots"].long()[:, None].expand(R, L)
    at = torch.arange(L, device=q.device)[None].expand(R, L)
    ok = at < s["past"][:, None]
    to[slot[ok], at[ok]] = s["mass"][slot[ok], at[ok]] + w[:, :L][ok]
    to[s["slots"].long()[:, None], s["past"][:, None] + torch.arange(n, device=q.device)] = w[:, L:]
    return to


def _plain_evict(s):
    case, slots = s["case"], s["slots"].long()
    B, bl = case["budget"], case["block"]
    R = slots.shape[0]
    n = s["hist"].long()[slots]
    i = torch.arange(s["cap"], device=slots.device)[None]
    m = s["mass"][slots]
    # always kept: the first rows and the last ones; never: rows past the end
    m = torch.where((i < case["sinks"]) | (i >= (n - case["recent"])[:, None]), math.inf, m)
    m = torch.where(i < n[:, None], m, -math.inf)
    order = torch.sort(m, dim=1, descending=True, stable=True).indices[:, :B]
    if order.shape[1] < B:
        order = torch.cat([order, order.new_full((R, B - order.shape[1]), s["cap"])], 1)
    order = torch.where(torch.arange(B, device=slots.device) < n[:, None], order, s["cap"]).sort(1).values
    live = order < s["cap"]
    kept = torch.where(live, order, -1)
    src = s["table"].long().view(-1, s["width"])[slots[:, None], kept.clamp(min=0) // bl] * bl + kept.clamp(min=0) % bl
    j = torch.arange(B, device=slots.device)[None].expand(R, B)
    dst = s["to"].long().view(-1, s["width"])[slots[:, None], (j // bl).clamp(max=s["width"] - 1)] * bl + j % bl
    for name in ("k", "v"):
        s["dst_" + name][dst[live]] = s["p" + name][src[live]]
    who = slots[:, None].expand(R, B)
    s["mass_out"][who[live], j[live]] = s["mass"][who[live], kept[live]]
    s["kept"].copy_(kept)
    return s["kept"], _value(s, s["dst_k"]), _value(s, s["dst_v"]), s["mass_out"]


def _positive(x):
    return torch.where(x > 0, x, 0.0)


def _plain_verify(s):
    """All requests walk down together: at each token its drafted continuations are tried in turn."""
    case, tok = s["case"], s["tokens"].long()
    R = s["tail"].shape[0]
    at = s["tail"].clone()
    r = torch.arange(R, device=at.device)
    n_accept = torch.zeros(R, dtype=torch.int64, device=at.device)
    s["path"].fill_(-1)
    walking = torch.ones(R, dtype=torch.bool, device=at.device)
    for _ in range(s["levels"]):
        p = _positive(s["target"][at].double())
        q = _positive(s["draft"][at].double()) if case["sampled"] else None
        c = torch.zeros(R, dtype=torch.float64, device=at.device)
        mass = torch.ones(R, dtype=torch.float64, device=at.device)
        rest = p.clone()
        down = torch.full_like(at, -1)
        for i in range(s["kids"].shape[1]):
            kid = s["kids"][at, i]
            ask = walking & (kid >= 0) & (down < 0)
            x = tok[kid.clamp(min=0)]
            u = s["u"][kid.clamp(min=0)].double()
            if case["sampled"]:
                yes = ask & (u * q[r, x] * mass < _positive(p[r, x] - c * q[r, x]))
                no = ask & ~yes
                c = torch.where(no, c + mass, c)
                rest = torch.where(no[:, None], _positive(p - c[:, None] * q), rest)
                mass = torch.where(no, rest.sum(1), mass)
            else:
                yes = ask & (u * mass < rest[r, x])
                no = ask & ~yes
                mass = torch.where(no, mass - rest[r, x], mass)
                rest[r, x] = torch.where(no, 0.0, rest[r, x])
            down = torch.where(yes, kid, down)
        stop = walking & (down < 0)
        # those that stop here draw their next token from what is left
        use = torch.where((rest.sum(1) > 0)[:, None], rest, p)
        cum = use.cumsum(1)
        aim = s["u_next"].double() * cum[:, -1]
        pick = torch.searchsorted(cum, aim[:, None], right=True)[:, 0]
        last = case["V"] - 1 - (use.flip(1) > 0).long().argmax(1)
        pick = torch.where(cum[:, -1] > 0, torch.minimum(pick, last), -1)
        s["next_token"].copy_(torch.where(stop, pick, s["next_token"]))
        go = walking & (down >= 0)
        s["path"][(s["first"] + n_accept)[go]] = down[go].int()
        n_accept += go
        at = torch.where(go, down, at)
        walking = go
    s["n_accept"].copy_(n_accept)
    return s["n_accept"], s["next_token"], s["path"]


# ---- 64 bits, one request at a time ---------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "draft": _exact_draft, "mass": _exact_mass, "evict": _exact_evict,
            "verify": _exact_verify}[case["op"]](case, s)


def _exact_rope(case, s):
    """Each pair as a complex number turned by exp(i p f)."""
    n, got = case["rot"] // 2, []
    turn = torch.polar(torch.full((len(s["pos"]), n), s["mscale"], dtype=torch.float64, device=DEV),
                       torch.outer((s["pos"] + s["offset"].long()[s["req"]]).double(), s["freqs"]))
    for x in (s["q"], s["k"]):
        y = x.double()
        pair = y[..., :2 * n].reshape(*y.shape[:-1], n, 2) if case["inter"] \
            else y[..., :2 * n].reshape(*y.shape[:-1], 2, n).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None])
        y[..., :2 * n] = (z if case["inter"] else z.transpose(-1, -2)).flatten(-2)
        got.append(y)
    return got


def _wide(s, x, which):
    return x.double() if s["descale"] is None else x.view(torch.float8_e4m3fn).double() * s["descale"][which].double()


def _exact_draft(case, s):
    G = case["Hq"] // case["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    for r, n in enumerate(s["lens"]):
        t = s["toks"][r][s["toks"][r] >= 0]
        row = s["rows"][r, :n]
        hide = torch.zeros(len(t), n + len(t), dtype=torch.bool, device=DEV)
        hide[:, n:] = ~s["see"][r, :len(t), :len(t)]
        for h in range(case["Hkv"]):
            k = torch.cat([_wide(s, s["pk"][row, h], 1), _wide(s, s["k"][t, h], 1)])
            v = torch.cat([_wide(s, s["pv"][row, h], 2), _wide(s, s["v"][t, h], 2)])
            for a in range(h * G, (h + 1) * G):
                x = (_wide(s, s["q"][t, a], 0) @ k.T * s["scale"]).masked_fill(hide, -math.inf)
                lse[t, a] = torch.logsumexp(x, 1)
                out[t, a] = torch.softmax(x, 1) @ v
    return out, lse


def _exact_mass(case, s):
    G = case["Hq"] // case["Hkv"]
    to = s["mass"].double()
    lse = s["lse"].double()
    for r, n in enumerate(s["lens"]):
        t, slot = s["roots"][r], int(s["slots"][r])
        add = torch.zeros(n + len(t), dtype=torch.float64, device=DEV)
        for a in range(case["Hq"]):
            k = torch.cat([_wide(s, s["pk"][s["rows"][r, :n], a // G], 1), _wide(s, s["k"][t, a // G], 1)])
            w = torch.exp(k @ _wide(s, s["q"][t, a], 0).T * s["scale"] - lse[t, a])
            w[n:] *= torch.ones(len(t), len(t), dtype=torch.float64, device=DEV).triu()
            add += w.sum(1)
        to[slot, :n] += add[:n]
        to[slot, n:n + len(t)] = add[n:]
    return to


def _exact_evict(case, s):
    """The rows are copied as they are: what is computed is which ones."""
    mass, slots = s["mass"].double().cpu().numpy(), s["slots"].cpu().numpy()
    bl, table, to = case["block"], s["table"].view(-1, s["width"]).cpu().numpy(), s["to"].view(-1, s["width"]).cpu().numpy()
    dk, dv, mo = s["dst_k"].clone(), s["dst_v"].clone(), np.zeros_like(mass)
    kept = np.full((case["R"], case["budget"]), -1, np.int64)
    for r, n in enumerate(s["lens"]):
        keep = set(range(n))
        if n > case["budget"]:
            keep = set(range(min(case["sinks"], n))) | set(range(max(0, n - case["recent"]), n))
            rest = sorted((i for i in range(n) if i not in keep), key=lambda i: (-mass[slots[r], i], i))
            keep |= set(rest[:case["budget"] - len(keep)])
        i = np.asarray(sorted(keep), np.int64)
        j = np.arange(len(i))
        kept[r, :len(i)] = i
        src, dst = table[slots[r], i // bl] * bl + i % bl, to[slots[r], j // bl] * bl + j % bl
        dk[_dev(dst)], dv[_dev(dst)] = s["pk"][_dev(src)], s["pv"][_dev(src)]
        mo[slots[r], j] = mass[slots[r], i]
    wide = lambda x: _value(s, x).double()  # noqa: E731
    return torch.from_numpy(kept).int(), wide(dk), wide(dv), torch.from_numpy(mo)


def _exact_verify(case, s):
    """No output is a computed number: tokens, rows and counts."""
    return None
