"""Host side of the speculative decoding operators, on the CPU: frequencies, the pool's
truncation, and every refusal before a device call (the addresses are fake, nothing
dereferences them)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tree_forked_decision_b200 import flide
from tree_forked_decision_b200.history import HistoryStore

A, B, NUL = 1 << 20, (1 << 20) + (1 << 16), None
S, C, I = flide.ERR_SHAPE, flide.ERR_CAPACITY, flide.ERR_INVALID

fake = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses: runs only where no device exists")


@pytest.fixture(scope="module")
def lib():
    return flide.load()


# ---- frequencies ----

def _freqs(rot, **kw):
    f, m = flide.rope_freqs(rot, device="cpu", **kw)
    return f.numpy(), m


def test_rope_frequencies():
    plain, m = _freqs(64)
    assert m == 1.0 and plain.shape == (32,) and plain[0] == 1.0
    # powers with 64-bit exponents: a few steps of 64 bits
    assert np.allclose(plain, 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    assert np.allclose(_freqs(64, scaling="linear", factor=4.0)[0], plain / 4, rtol=1e-15)
    ntk, m = _freqs(64, scaling="ntk", factor=4.0)
    # the fastest pair is kept, the slowest turns 4 times slower
    assert m == 1.0 and ntk[0] == 1.0 and math.isclose(ntk[-1], plain[-1] / 4, rel_tol=1e-12)
    yarn, m = _freqs(64, scaling="yarn", factor=4.0, orig_len=4096)
    assert math.isclose(m, 0.1 * math.log(4) + 1, rel_tol=2.0 ** -23)
    turns = 4096 * plain / (2 * math.pi)
    assert np.array_equal(yarn[turns >= 32], plain[turns >= 32])
    assert np.allclose(yarn[turns <= 1], plain[turns <= 1] / 4, rtol=1e-15)
    between = (turns > 1) & (turns < 32)
    assert between.any() and np.all((yarn[between] < plain[between]) & (yarn[between] > plain[between] / 4))
    assert _freqs(2, scaling="ntk", factor=4.0)[0].tolist() == [1.0]


@pytest.mark.parametrize("kw,code", [
    (dict(rot=0), S), (dict(rot=3), S), (dict(rot=1026), S), (dict(scaling=4), S), (dict(scaling=-1), S),
    (dict(base=0.0), I), (dict(base=-1.0), I), (dict(base=math.nan), I), (dict(base=math.inf), I),
    (dict(scaling=1, factor=0.5), I), (dict(scaling=2, factor=math.nan), I), (dict(scaling=3, orig_len=0.0), I),
    (dict(scaling=3, fast=1.0), I), (dict(scaling=3, slow=-1.0), I), (dict(scaling=3, fast=math.inf), I),
    (dict(scaling=1, factor=math.inf), I),
])
def test_rope_freqs_refusals(lib, kw, code):
    a = dict(rot=64, base=10000.0, scaling=0, factor=2.0, orig_len=4096.0, fast=32.0, slow=1.0)
    a.update(kw)
    buf, m = (ctypes.c_double * 1024)(), ctypes.c_float()
    assert lib.flide_rope_freqs(a["rot"], a["base"], a["scaling"], a["factor"], a["orig_len"], a["fast"], a["slow"],
                                buf, ctypes.byref(m)) == code
    assert lib.flide_rope_freqs(64, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, None, ctypes.byref(m)) == S
    assert lib.flide_rope_freqs(64, 10000.0, 0, 1.0, 0.0, 0.0, 0.0, buf, None) == S
    with pytest.raises(ValueError):
        flide.rope_freqs(64, scaling="cubic", device="cpu")


# ---- pool ----

def test_pool_truncate(lib):
    pool = lib.flide_pool_create(8, 16, 2, 6)
    try:
        assert lib.flide_pool_append(pool, 0, 70) == 0 and lib.flide_pool_append(pool, 1, 20) == 0
        table, length = (ctypes.c_int32 * 12)(), (ctypes.c_int32 * 2)()
        lib.flide_pool_export(pool, table, length)
        before = list(table)
        assert lib.flide_pool_free_blocks(pool) == 1
        for slot, rows in ((2, 0), (-1, 0), (0, 71), (0, -1)):
            assert lib.flide_pool_truncate(pool, slot, rows) == I
        assert lib.flide_pool_truncate(NUL, 0, 0) == I
        assert lib.flide_pool_truncate(pool, 0, 33) == flide.OK
        assert lib.flide_pool_length(pool, 0) == 33 and lib.flide_pool_free_blocks(pool) == 3
        lib.flide_pool_export(pool, table, length)
        assert list(table)[:6] == before[:3] + [-1] * 3 and list(table)[6:] == before[6:]
        assert list(length) == [33, 20]
        assert lib.flide_pool_truncate(pool, 0, 33) == flide.OK  # nothing more to cut
        assert lib.flide_pool_append(pool, 0, 48) == 33
        assert lib.flide_pool_truncate(pool, 0, 0) == flide.OK and lib.flide_pool_free_blocks(pool) == 6
    finally:
        lib.flide_pool_destroy(pool)


def test_store_bookkeeping():
    store = HistoryStore(n_blocks=4, block_rows=16, max_requests=2, max_blocks=3, Hkv=1, d=8, device="cpu")
    assert store.pos_offset([1, -1, 0]).tolist() == [0, 0, 0]
    with pytest.raises(ValueError):
        store.evict([0], 4)  # no weights yet
    with pytest.raises(ValueError):
        store.evict([0, 0], 4)
    with pytest.raises(ValueError):
        store.accumulate_mass(None, None, None, None, 1.0, [1, 1])
    store.mass = torch.ones(2, 48)
    store.evicted_h[1] = 7
    assert store.pos_offset([1, -1]).tolist() == [7, 0]
    store.release(1)
    assert store.pos_offset([1]).tolist() == [0]
    assert bool((store.mass[0] == 1).all()) and bool((store.mass[1] == 0).all())  # the slot starts over


# ---- refusals of the device entry points ----

def _idx(R=2, N=5, T=64, max_depth=2):
    x = flide.TreeIndexC()
    x.R, x.N, x.T, x.max_depth = R, N, T, max_depth
    for i, name in enumerate(flide.INDEX_ARRAYS):
        setattr(x, name, A + 256 * i)
    x.work_len = 1 << 12
    return ctypes.byref(x)


@fake
@pytest.mark.parametrize("kw,code", [
    (dict(idx=NUL), S), (dict(freqs=NUL), S), (dict(q=NUL), S), (dict(qo=NUL), S), (dict(ko=NUL), S),
    (dict(q=NUL, qo=NUL, k=NUL, ko=NUL), S), (dict(Hq=0), S), (dict(Hkv=-1), S), (dict(d=0), S), (dict(rot=0), S),
    (dict(rot=7), S), (dict(rot=130), S), (dict(d=2000, rot=1026), S), (dict(dtype=flide.E4M3), S), (dict(dtype=9), S),
    (dict(idx=_idx(T=-1)), S), (dict(Hq=1 << 20, d=1 << 12), C), (dict(idx=_idx(T=0)), flide.OK),
])
def test_rope_refusals(lib, kw, code):
    a = dict(idx=_idx(), freqs=A, q=A, k=A, qo=B, ko=B, Hq=16, Hkv=4, d=128, rot=128, dtype=flide.BF16)
    a.update(kw)
    assert lib.flide_rope(a["idx"], NUL, a["freqs"], a["q"], a["k"], a["qo"], a["ko"], a["Hq"], a["Hkv"], a["d"],
                          a["rot"], 0, 0, 1.0, a["dtype"], NUL) == code


DRAFT = [
    (dict(idx=NUL), S), (dict(q=NUL), S), (dict(out=NUL), S), (dict(ws=NUL), S), (dict(Hq=0), S), (dict(Hkv=0), S),
    (dict(Hq=12, Hkv=8), S), (dict(d=16), S), (dict(d=100), S), (dict(d=288), S), (dict(dtype=7), S),
    (dict(dtype=flide.E4M3), S), (dict(dtype=flide.E4M3, descale=A, d=64), S), (dict(idx=_idx(R=-1)), S),
    (dict(idx=_idx(T=-1)), S), (dict(idx=_idx(R=4097)), C), (dict(idx=_idx(T=1 << 28)), C), (dict(ws_bytes=100), C),
    (dict(ws=A + 16), S), (dict(q=A + 8), S), (dict(out=B + 8), S), (dict(scale=-0.1), I),
    (dict(scale=math.nan), I), (dict(scale=math.inf), I), (dict(idx=_idx(T=0)), flide.OK), (dict(idx=_idx(R=0)), flide.OK),
]


@fake
@pytest.mark.parametrize("kw,code", DRAFT + [(dict(past=NUL), S), (dict(past_rows=-1), S)])
def test_draft_attn_refusals(lib, kw, code):
    a = dict(idx=_idx(), q=A, past=A, past_rows=10, Hq=16, Hkv=4, d=128, dtype=flide.BF16, descale=NUL, out=B, ws=A,
             ws_bytes=1 << 40, scale=0.1)
    a.update(kw)
    assert lib.flide_draft_attn(a["q"], A, A, a["past"], A, a["past_rows"], a["idx"], a["Hq"], a["Hkv"], a["d"],
                                a["dtype"], a["descale"], a["scale"], a["out"], NUL, a["ws"], a["ws_bytes"], NUL) == code


PAGED = [(dict(pool=NUL), S), (dict(table=NUL), S), (dict(slot=NUL), S), (dict(n_blocks=0), S), (dict(max_blocks=0), S),
         (dict(n_slots=0), S), (dict(block_rows=0), S), (dict(block_rows=24), S), (dict(block_rows=-16), S)]


@fake
@pytest.mark.parametrize("kw,code", DRAFT + PAGED)
def test_draft_attn_paged_refusals(lib, kw, code):
    a = dict(idx=_idx(), q=A, pool=A, table=A, slot=A, n_blocks=4, block_rows=16, max_blocks=2, n_slots=2, Hq=16, Hkv=4,
             d=128, dtype=flide.BF16, descale=NUL, out=B, ws=A, ws_bytes=1 << 40, scale=0.1)
    a.update(kw)
    assert lib.flide_draft_attn_paged(a["q"], A, A, a["pool"], A, a["n_blocks"], a["block_rows"], a["table"],
                                      a["max_blocks"], a["slot"], a["n_slots"], a["idx"], a["Hq"], a["Hkv"], a["d"],
                                      a["dtype"], a["descale"], a["scale"], a["out"], NUL, a["ws"], a["ws_bytes"], NUL) == code


@fake
@pytest.mark.parametrize("kw,code", [x for x in DRAFT if not {"out", "ws", "ws_bytes", "scale"} & set(x[0])
                                     and "q" not in x[0] and x[1] != C] + PAGED
                         + [(dict(q=NUL), S), (dict(lse=NUL), S), (dict(mass=NUL), S), (dict(idx=_idx(R=4097)), C)])
def test_history_mass_refusals(lib, kw, code):
    a = dict(idx=_idx(), q=A, lse=A, pool=A, table=A, slot=A, n_blocks=4, block_rows=16, max_blocks=2, n_slots=2, Hq=16,
             Hkv=4, d=128, dtype=flide.BF16, descale=NUL, mass=A)
    a.update(kw)
    assert lib.flide_history_mass(a["q"], A, a["lse"], a["pool"], a["n_blocks"], a["block_rows"], a["table"],
                                  a["max_blocks"], a["slot"], a["n_slots"], a["idx"], a["Hq"], a["Hkv"], a["d"],
                                  a["dtype"], a["descale"], 0.1, a["mass"], B, NUL) == code


@fake
@pytest.mark.parametrize("kw,code", [
    (dict(slot=NUL), S), (dict(pool=NUL), S), (dict(mass=NUL), S), (dict(kept=NUL), S), (dict(R=-1), S),
    (dict(n_slots=0), S), (dict(block_rows=0), S), (dict(n_blocks=0), S), (dict(dst_blocks=0), S), (dict(Hkv=0), S),
    (dict(budget=0), S), (dict(sinks=-1), S), (dict(recent=-1), S), (dict(sinks=60, recent=41), S),
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), S), (dict(dtype=5), S), (dict(Hkv=1, d=4), S),
    (dict(Hkv=1 << 13, d=128), S), (dict(pool=A + 8), S), (dict(n_blocks=1 << 26), C), (dict(R=4097), C), (dict(max_blocks=1 << 20, block_rows=1 << 12), C),
    (dict(R=0), flide.OK),
])
def test_history_evict_refusals(lib, kw, code):
    a = dict(R=2, slot=A, n_slots=3, max_blocks=4, block_rows=64, pool=A, n_blocks=8, Hkv=2, d=128, dtype=flide.BF16,
             mass=A, budget=100, sinks=4, recent=10, dst_blocks=8, kept=B)
    a.update(kw)
    assert lib.flide_history_evict(a["R"], a["slot"], a["n_slots"], A, A, a["max_blocks"], a["block_rows"], a["pool"],
                                   A, a["n_blocks"], a["Hkv"], a["d"], a["dtype"], a["mass"], a["budget"], a["sinks"],
                                   a["recent"], A, A, A, a["dst_blocks"], A, a["kept"], A, NUL) == code


@fake
@pytest.mark.parametrize("kw,code", [
    (dict(idx=NUL), S), (dict(tokens=NUL), S), (dict(target=NUL), S), (dict(path=NUL), S), (dict(V=0), S),
    (dict(V=(1 << 26) + 1), S), (dict(dtype=flide.E4M3), S), (dict(idx=_idx(R=-1)), S),
    (dict(idx=_idx(R=(1 << 24) + 1)), C), (dict(idx=_idx(R=0)), flide.OK),
])
def test_verify_refusals(lib, kw, code):
    a = dict(idx=_idx(), tokens=A, target=A, V=100, dtype=flide.F32, path=B)
    a.update(kw)
    assert lib.flide_verify_draft(a["idx"], a["tokens"], a["target"], NUL, A, A, a["V"], a["dtype"], B, B, a["path"],
                                  NUL) == code


def test_workspace_bytes(lib):
    f = lib.flide_draft_attn_workspace_bytes
    assert f(-1, 4, 8, 2, 128) == 0 and f(1, 4, 8, 3, 128) == 0 and f(1, 4, 0, 1, 128) == 0 and f(1, 4, 8, 2, 0) == 0
    assert 0 < f(8, 8, 8, 2, 128) < f(8, 64, 8, 2, 128) < f(8, 640, 8, 2, 128)


# ---- the binding's own checks: host tensors, types and shapes never reach the library ----

class _Index:
    R, T, N, c = 1, 4, 3, flide.TreeIndexC()
    buf = torch.zeros(1)


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_checks():
    q, k, f = _t(4, 8, 64), _t(4, 2, 64), torch.zeros(32, dtype=torch.float64)
    ix, i32 = _Index(), torch.zeros(4, dtype=torch.int32)
    lse, ws = _t(4, 8, dtype=torch.float32), _t(64, dtype=torch.uint8)
    for bad in (lambda: flide.rope(q, k, ix, f), lambda: flide.rope(None, None, ix, f),
                lambda: flide.rope(q[:3], k[:3], ix, f), lambda: flide.rope(q, _t(5, 2, 64), ix, f),
                lambda: flide.rope(q, k, ix, f, pos_offset=i32[:0]),
                lambda: flide.rope(q, k, ix, f, q_out=_t(4, 8, 32), k_out=k),
                lambda: flide.draft_attn(q, k, k, ix, 1.0, past_k=k, out=q, lse=lse, workspace=ws),
                lambda: flide.draft_attn(q, k, k, ix, 1.0, past_k=_t(4, 2, 32), past_v=_t(4, 2, 32)),
                lambda: flide.draft_attn(q, k, k, ix, 1.0, out=q, lse=lse, workspace=ws),  # host tensors
                lambda: flide.draft_attn(q, k, k, ix, 1.0, out=q, lse=lse[:2], workspace=ws),
                lambda: flide.draft_attn_paged(q, k, k, ix, 1.0, k, k, i32, i32[:0], 16, 1, out=q, lse=lse, workspace=ws),
                lambda: flide.verify_draft(ix, i32, _t(3, 9, dtype=torch.float32), lse[0], lse[0]),
                lambda: flide.verify_draft(ix, i32[:2], _t(4, 9, dtype=torch.float32), lse[0], lse[0]),
                lambda: flide.history_mass(q, k, lse, ix, 1.0, k, i32, i32, 16, 4, _t(1, 65, dtype=torch.float32)),
                lambda: flide.history_evict(i32, i32, i32, 16, 1, k, k, _t(4, 16, dtype=torch.float32), 2, i32, dst_k=k),
                lambda: flide.history_evict(i32, i32, i32[:2], 16, 1, k, k, _t(4, 16, dtype=torch.float32), 2, i32),
                lambda: flide.history_evict(i32, i32, i32, 16, 1, k, k, _t(4, 16, dtype=torch.float32), 0, i32)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: flide.rope(q, _t(4, 2, 64, dtype=torch.float32), ix, f),
                lambda: flide.rope(q, k, ix, f.float()), lambda: flide.rope(q, k, ix, f, pos_offset=i32.long()),
                lambda: flide.rope(q.half(), k.half(), ix, f.float(), q_out=q.half(), k_out=k.half()),
                lambda: flide.rope(q, k, ix, f, q_out=q.float(), k_out=k),
                lambda: flide.draft_attn(q, k.float(), k.float(), ix, 1.0),
                lambda: flide.draft_attn(q, k, k, ix, 1.0, descale=lse[0]),
                lambda: flide.draft_attn(q.to(torch.uint8), k.to(torch.uint8), k.to(torch.uint8), ix, 1.0),
                lambda: flide.draft_attn(q, k, k, ix, 1.0, out=q.float(), lse=lse, workspace=ws),
                lambda: flide.verify_draft(ix, i32, _t(4, 9), lse[0], lse[0], draft=_t(4, 9, dtype=torch.float32)),
                lambda: flide.verify_draft(ix, i32.long(), _t(4, 9), lse[0], lse[0]),
                lambda: flide.history_mass(q, k, lse, ix, 1.0, k, i32, i32, 16, 4, _t(1, 64)),
                lambda: flide.history_evict(i32, i32, i32, 16, 1, k, k.float(), _t(4, 16, dtype=torch.float32), 2, i32)):
        with pytest.raises(TypeError):
            bad()
