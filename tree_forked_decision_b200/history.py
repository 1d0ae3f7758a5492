"""Multi-step agent history in a block-paged checkpoint pool.

An agent takes decision after decision on a growing history: each step's root
(the new observation) is appended to what came before, and the next step
resumes from it, so the shared prefix is computed once over the whole episode
(kongchang.com article on Flide, closing section: growing agent histories and
checkpoint reuse; techfi24.com, "Exact State Forking").

``HistoryStore`` owns the device pool -- K/V history rows in blocks of
``block_rows`` rows and one fp32 GDN state per request slot -- and the native
block allocator (``flide_pool_*`` in libflide.so).  Per step:

    past_len, past_k, past_v, state_in = store.resume(slots)       # before
    ... flide_tree_build / fork_attn / fork_gdn on the step's tree ...
    store.commit(slots, index, k, v, node_state)                    # after

``resume`` packs each slot's history as the batch's past rows and GDN
state_in; ``commit`` reserves blocks for each request's root tokens on the
host, copies the block table to the device, and appends the root rows and the
root's end state.  ``release(slot)`` returns a finished request's blocks.

Without the packed copy (block_rows a multiple of 128):

    past_len, state_in = store.resume_lengths(slots)
    ... flide_tree_build ...
    o = store.fork_attn_paged(q, k, v, index, scale, slots)   # past read in place

A speculative decoding step (a root of committed tokens and drafted tokens below
it), with the history bounded to `budget` rows:

    past_len, state_in = store.resume_lengths(slots)
    ... flide_tree_build; flide.rope(q, k, index, freqs, pos_offset=store.pos_offset(slots)) ...
    o, lse = store.draft_attn(q, k, v, index, scale, slots)
    n, token, path = flide.verify_draft(index, tokens, target, u, u_next, draft=draft)
    store.accumulate_mass(q, k, lse, index, scale, slots)     # before commit
    store.commit(slots, tree, index, k, v, node_state)
    store.evict(slots, budget, sinks=4, recent=64)

The store's calls take the slots from the host and copy them to the device each time;
a step that is captured into a CUDA graph calls ``flide.draft_attn_paged`` and
``flide.history_mass`` with the store's ``pool_k``, ``pool_v``, ``table`` and ``mass`` (there
from the first ``accumulate_mass`` on), and slots and a workspace of its own.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import flide


class HistoryStore:
    def __init__(self, n_blocks: int, block_rows: int, max_requests: int, max_blocks: int,
                 Hkv: int, d: int, H: int = 0, dk: int = 0, dv: int = 0,
                 dtype=torch.bfloat16, device="cuda"):
        lib = flide._lib()
        self._lib = lib
        self._pool = lib.flide_pool_create(n_blocks, block_rows, max_requests, max_blocks)
        if not self._pool:
            raise flide.FlideError(flide.ERR_SHAPE, "flide_pool_create")
        self.n_blocks, self.block_rows = n_blocks, block_rows
        self.max_requests, self.max_blocks = max_requests, max_blocks
        self.Hkv, self.d, self.H, self.dk, self.dv = Hkv, d, H, dk, dv
        self.dtype, self.device = dtype, device
        self.pool_k = torch.zeros((n_blocks * block_rows, Hkv, d), dtype=dtype, device=device)
        self.pool_v = torch.zeros_like(self.pool_k)
        self.pool_S = (torch.zeros((max_requests, H, dv, dk), dtype=torch.float32, device=device)
                       if H else None)
        self.table_h = np.full(max_requests * max_blocks, -1, np.int32)
        self.len_h = np.zeros(max_requests, np.int32)
        self.table = torch.full((max_requests * max_blocks,), -1, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(max_requests, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.mass = None  # attention weight per history row, from accumulate_mass on
        self.evicted_h = np.zeros(max_requests, np.int32)  # rows evicted per slot
        self._weighed = {}  # slot -> its rows' weights before a step that is not committed yet

    def __del__(self):
        pool = getattr(self, "_pool", None)
        if pool:
            self._lib.flide_pool_destroy(pool)
            self._pool = None

    # -- host bookkeeping ---------------------------------------------------
    def length(self, slot: int) -> int:
        return int(self._lib.flide_pool_length(self._pool, slot))

    def free_blocks(self) -> int:
        return int(self._lib.flide_pool_free_blocks(self._pool))

    def release(self, slot: int):
        flide._check(self._lib.flide_pool_release(self._pool, slot), "flide_pool_release")
        self.evicted_h[slot] = 0
        self._weighed.pop(slot, None)
        if self.mass is not None:
            self.mass[slot].zero_()
        self._sync_table()

    def _sync_table(self):
        flide._check(self._lib.flide_pool_export(self._pool, self.table_h.ctypes.data_as(ctypes.c_void_p),
                                                 self.len_h.ctypes.data_as(ctypes.c_void_p)),
                     "flide_pool_export")
        self.table.copy_(torch.from_numpy(self.table_h))
        self.lengths.copy_(torch.from_numpy(self.len_h))

    # -- device steps -------------------------------------------------------
    def resume(self, slots, past_rows: int | None = None):
        """Past rows, lengths and GDN state_in for a batch whose request r
        continues slot slots[r] (-1: no history)."""
        slots = [int(s) for s in slots]
        R = len(slots)
        rows = sum(int(self.len_h[s]) for s in slots if s >= 0)
        past_rows = max(rows, 1) if past_rows is None else past_rows
        req = torch.tensor(slots, dtype=torch.int32, device=self.device)
        past_len = torch.zeros(R, dtype=torch.int32, device=self.device)
        pk = torch.empty((past_rows, self.Hkv, self.d), dtype=self.dtype, device=self.device)
        pv = torch.empty_like(pk)
        state_in = (torch.empty((R, self.H, self.dv, self.dk), dtype=torch.float32, device=self.device)
                    if self.H else None)
        self.status.zero_()
        flide._check(self._lib.flide_history_gather(
            R, flide._ptr(req), self.max_requests, flide._ptr(self.lengths), flide._ptr(self.table),
            self.max_blocks, self.block_rows, flide._ptr(self.pool_k), flide._ptr(self.pool_v),
            self.Hkv, self.d, flide._dtype_code(self.pool_k), flide._ptr(self.pool_S), self.H,
            self.dk, self.dv, flide._ptr(past_len), flide._ptr(pk), flide._ptr(pv), past_rows,
            flide._ptr(state_in), flide._ptr(self.status), flide._stream()), "flide_history_gather")
        return past_len, pk, pv, state_in

    def resume_lengths(self, slots):
        """past_len and GDN state_in for a batch whose request r continues
        slot slots[r] (-1: no history), without packing the rows: for
        fork_attn_paged, which reads them in place."""
        slots = [int(s) for s in slots]
        R = len(slots)
        req = torch.tensor(slots, dtype=torch.int32, device=self.device)
        past_len = torch.zeros(R, dtype=torch.int32, device=self.device)
        state_in = (torch.empty((R, self.H, self.dv, self.dk), dtype=torch.float32, device=self.device)
                    if self.H else None)
        self.status.zero_()
        flide._check(self._lib.flide_history_gather(
            R, flide._ptr(req), self.max_requests, flide._ptr(self.lengths), flide._ptr(self.table),
            self.max_blocks, self.block_rows, flide._ptr(self.pool_k), flide._ptr(self.pool_v),
            self.Hkv, self.d, flide._dtype_code(self.pool_k), flide._ptr(self.pool_S), self.H,
            self.dk, self.dv, flide._ptr(past_len), None, None, 0, flide._ptr(state_in),
            flide._ptr(self.status), flide._stream()), "flide_history_gather")
        return past_len, state_in

    def fork_attn_paged(self, q, k, v, index: flide.TreeIndex, scale: float, slots, out=None):
        """Fork attention of a batch whose request r continues slot slots[r],
        the past rows read in place from this pool's blocks."""
        req = torch.tensor([int(s) for s in slots], dtype=torch.int32, device=self.device)
        return flide.fork_attn_paged(q, k, v, index, scale, self.pool_k, self.pool_v, self.table,
                                     req, self.block_rows, self.max_blocks, out=out)

    def draft_attn(self, q, k, v, index: flide.TreeIndex, scale: float, slots, out=None, lse=None,
                   workspace=None):
        """fork_attn_paged for a few tokens per request over long histories (blocks of
        any multiple of 16 rows); also returns the log-sum-exp [T, Hq]."""
        req = torch.tensor([int(s) for s in slots], dtype=torch.int32, device=self.device)
        return flide.draft_attn_paged(q, k, v, index, scale, self.pool_k, self.pool_v, self.table, req,
                                      self.block_rows, self.max_blocks, out=out, lse=lse,
                                      workspace=workspace)

    def pos_offset(self, slots):
        """Rows evicted from each request's history (int32 [R], device): what its
        positions are ahead of its past length, for flide.rope."""
        off = [int(self.evicted_h[s]) if s >= 0 else 0 for s in (int(s) for s in slots)]
        return torch.tensor(off, dtype=torch.int32, device=self.device)

    def accumulate_mass(self, q, k, lse, index: flide.TreeIndex, scale: float, slots):
        """Adds the attention weight that this step's root tokens gave each history row,
        and starts that of the root's own rows: after draft_attn, before commit.  A commit
        that is refused takes it back (a step's retry weighs its rows again)."""
        slots = self._once(slots, "accumulate_mass")
        if self.mass is None:
            self.mass = torch.zeros((self.max_requests, self.max_blocks * self.block_rows),
                                    dtype=torch.float32, device=self.device)
        req = torch.tensor(slots, dtype=torch.int32, device=self.device)
        live = [s for s in slots if s >= 0]
        rows = max((self.length(s) for s in live), default=0)
        before = dict(zip(live, self.mass[:, :rows][live]))
        flide.history_mass(q, k, lse, index, scale, self.pool_k, self.table, req, self.block_rows,
                           self.max_blocks, self.mass)
        self._weighed.update(before)

    def evict(self, slots, budget: int, sinks: int = 0, recent: int = 0):
        """Cuts the histories of `slots` that are longer than `budget` rows down to their
        first `sinks`, last `recent` and heaviest rows, in place, and frees the blocks
        past them.  Returns the rows kept, int32 [len(slots), budget], -1 past the end."""
        slots = self._once(slots, "evict")
        if self.mass is None:
            raise ValueError("evict needs the rows' attention weight (accumulate_mass)")
        req = torch.tensor(slots, dtype=torch.int32, device=self.device)
        kept = flide.history_evict(req, self.lengths, self.table, self.block_rows, self.max_blocks,
                                   self.pool_k, self.pool_v, self.mass, int(budget), self.status,
                                   sinks=int(sinks), recent=int(recent))
        # (slots, lengths and blocks are the pool's own: nothing is left for the device to refuse)
        for s in slots:
            self._weighed.pop(s, None)  # its rows have moved
            if s >= 0 and self.length(s) > budget:
                self.evicted_h[s] += self.length(s) - budget
                self.mass[s, budget:].zero_()  # rows to come start without weight
                flide._check(self._lib.flide_pool_truncate(self._pool, s, int(budget)),
                             "flide_pool_truncate")
        self._sync_table()
        return kept

    def _once(self, slots, where):
        """The slots as ints, each one of the store's and at most once (-1: none)."""
        slots = [int(s) for s in slots]
        live = [s for s in slots if s >= 0]
        if len(set(live)) != len(live):
            raise ValueError("a slot may stand for one request of a call")
        if any(s >= self.max_requests for s in live):
            raise flide.FlideError(flide.ERR_INVALID, where)
        return slots

    def _take_back(self, weighed):
        """Puts back rows' weights from before a step (slot -> weights)."""
        for s, before in weighed.items():
            n = self.length(s)
            self.mass[s, :n] = before[:n]
            self.mass[s, n:].zero_()

    def reserve(self, slots, tree):
        """Host half of commit: reserves each request's root rows in its slot
        (all requests or none: on FlideError no slot changes, and the weights that
        accumulate_mass gave them for this step are taken back), refreshes the
        device block table and lengths, and returns the start rows (-1 where
        slots[r] is -1).  Each slot at most once per step (ValueError)."""
        slots = [int(s) for s in slots]
        kept = [s for s in slots if s >= 0]
        if len(set(kept)) != len(kept):
            raise ValueError("a slot may be continued by one request per step "
                             "(two end states would race for it)")
        rp, _parent, seg, _past = tree.arrays()
        counts = np.array([int(seg[rp[r]]) if rp[r + 1] > rp[r] else 0 for r in range(len(slots))],
                          np.int32)
        sl = np.array(slots, np.int32)
        start = np.zeros(len(slots), np.int32)
        p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
        weighed = {s: self._weighed.pop(s) for s in kept if s in self._weighed}
        code = self._lib.flide_pool_append_batch(self._pool, len(slots), p(sl), p(counts), p(start))
        if code != flide.OK:
            self._take_back(weighed)
        flide._check(code, "flide_pool_append_batch")
        self._sync_table()
        return start

    def commit(self, slots, tree, index: flide.TreeIndex, k, v, node_state=None):
        """Appends request r's root tokens (this step's observation) and its
        root's end GDN state to slot slots[r] (-1: nothing kept).  Where it raises, the
        store is as it was before the step."""
        slots = [int(s) for s in slots]
        weighed = {s: self._weighed[s] for s in slots if s in self._weighed}
        start = None
        try:
            # (rows of another type would be written past the pool's end)
            flide._rows_like("commit", self.pool_k, k=k, v=v)
            tokens = int(tree.arrays()[2].sum())
            if min(k.shape[0], v.shape[0]) < tokens:
                raise ValueError(f"commit: k and v need {tokens} rows, got {k.shape[0]} and {v.shape[0]}")
            if self.H:
                flide._states_like("commit", self.H, self.dv, self.dk, node_state=node_state)
            pk, pv, ps = flide._ptr(k), flide._ptr(v), flide._ptr(node_state if self.H else None)
            start = self.reserve(slots, tree)
            req = torch.tensor(slots, dtype=torch.int32, device=self.device)
            st_d = torch.from_numpy(start).to(self.device)
            flide._check(self._lib.flide_history_append(
                ctypes.byref(index.c), flide._ptr(req), flide._ptr(st_d), flide._ptr(self.table),
                self.max_blocks, self.block_rows, pk, pv, flide._ptr(self.pool_k),
                flide._ptr(self.pool_v), self.Hkv, self.d, flide._dtype_code(k), ps, self.H, self.dk,
                self.dv, flide._ptr(self.pool_S), flide._stream()), "flide_history_append")
        except Exception:
            if start is not None:  # the rows are reserved, but nothing stands in them
                for s, n in zip(slots, start):
                    if s >= 0:
                        self._lib.flide_pool_truncate(self._pool, s, int(n))
                self._sync_table()
            for s in weighed:
                self._weighed.pop(s, None)
            self._take_back(weighed)
            raise
