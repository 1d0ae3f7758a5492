"""Rotary positions against complex turns in 64 bits.

Tolerance: the fraction of a turn is rounded to 32 bits (at most 2^-26 of a turn,
9.4e-8 rad), sincospi is off by 2 steps (1.2e-7 each of cos and sin), products and
the sum by 3 roundings (1.8e-7): within 6e-7 m (|a| + |b|), then the output's own
rounding."""
import numpy as np
import pytest
import torch

from tree_forked_decision_b200 import flide, inputs

import decode_helpers as dh
from gpu_helpers import build

pytestmark = pytest.mark.gpu


def _want(x, pos, freqs, m, inter, transpose):
    n = freqs.shape[0]
    y = x.double().clone()
    pair = y[..., :2 * n].unflatten(-1, (n, 2)) if inter else y[..., :2 * n].unflatten(-1, (2, n)).transpose(-1, -2)
    pair = pair.contiguous()
    angle = torch.outer(torch.as_tensor(pos, dtype=torch.float64), freqs)
    turn = torch.polar(torch.full_like(angle, m), -angle if transpose else angle)
    z = torch.view_as_real(torch.view_as_complex(pair) * turn[:, None])
    size = pair.abs().sum(-1, keepdim=True).expand_as(pair) * m
    back = (lambda u: u.flatten(-2)) if inter else (lambda u: u.transpose(-1, -2).flatten(-2))
    y[..., :2 * n] = back(z)
    tol = torch.zeros_like(y)
    tol[..., :2 * n] = 6e-7 * back(size)
    return y, tol


CASES = [  # Hq, Hkv, d, rot, scaling
    (16, 4, 128, 128, "none"), (4, 4, 64, 32, "linear"), (5, 1, 80, 40, "ntk"), (8, 2, 128, 64, "yarn"),
    (3, 1, 6, 2, "ntk"), (2, 1, 1030, 1024, "none"), (1, 1, 33, 30, "yarn"),
]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", CASES, ids=[f"d{c[2]}r{c[3]}{c[4]}" for c in CASES])
def test_rope(case, dtype, inter):
    Hq, Hkv, d, rot, scaling = case
    tree = inputs._tree([(1000003, [(-1, 3), (0, 2), (0, 1)]), (0, []), (7, [(-1, 0), (0, 5)]), (0, [(-1, 1)])], 1)
    g = torch.Generator().manual_seed(d)
    spare = 3
    T = tree.T + spare
    q, k = (torch.randn(T, h, d, generator=g).to(dtype) for h in (Hq, Hkv))
    off = np.array([5, 6, 900, -0], np.int32)
    req, pos, _ = dh.layout(tree)
    freqs, m = flide.rope_freqs(rot, 10000.0, scaling, factor=4.0 if scaling != "none" else 1.0, orig_len=4096)
    _, idx = build(tree, T=T)
    for transpose in (False, True):
        qo, ko = (torch.full_like(x, 9.0).cuda() for x in (q, k))
        flide.rope(q.cuda(), k.cuda(), idx, freqs, pos_offset=torch.from_numpy(off).cuda(), mscale=m,
                   interleaved=inter, transpose=transpose, q_out=qo, k_out=ko)
        qi, ki = q.cuda(), k.cuda()
        assert flide.rope(qi, ki, idx, freqs, pos_offset=torch.from_numpy(off).cuda(), mscale=m,
                          interleaved=inter, transpose=transpose, q_out=qi, k_out=ki) == (qi, ki)
        torch.cuda.synchronize()
        for x, out, here in ((q, qo, qi), (k, ko, ki)):
            y, tol = _want(x[:tree.T], pos + off[req], freqs.cpu(), m, inter, transpose)
            err = (out[:tree.T].double().cpu() - y).abs()
            assert bool((err <= tol + dh.step(dtype) * y.abs()).all()), float(err.max())
            assert torch.equal(out[:tree.T, :, rot:].cpu(), x[:tree.T, :, rot:])  # copied
            assert bool((out[tree.T:] == 9).all())                                 # left as they were
            assert torch.equal(out[:tree.T], here[:tree.T]) and torch.equal(here[tree.T:].cpu(), x[tree.T:])


def test_one_tensor_and_no_offset():
    tree = inputs._tree([(12, [(-1, 4), (0, 2)])], 1)
    x = torch.randn(tree.T, 3, 64).cuda()
    freqs, m = flide.rope_freqs(64)
    _, idx = build(tree)
    a, none = flide.rope(x, None, idx, freqs)
    none2, b = flide.rope(None, x, idx, freqs, pos_offset=torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert none is None and none2 is None and torch.equal(a, b)


def test_gradient_is_the_transposed_turn():
    """Differences of <rope(x), g> along e equal <e, rope^T(g)>: rope is linear, so they are exact
    but for roundings (both sides 32 bits: 64 pairs of terms, 6e-7 each, twice)."""
    tree = inputs._tree([(5000, [(-1, 4), (0, 2)])], 1)
    g = torch.Generator().manual_seed(1)
    x, e, w = (torch.randn(tree.T, 2, 64, generator=g).cuda() for _ in range(3))
    freqs, m = flide.rope_freqs(64, scaling="yarn", factor=8.0, orig_len=1024)
    _, idx = build(tree)
    turn = lambda y, t=False: flide.rope(y, None, idx, freqs, mscale=m, transpose=t)[0].double()  # noqa: E731
    grad = turn(w, True)
    left = ((turn(x + e) - turn(x - e)) / 2 * w.double()).sum()
    right = (e.double() * grad).sum()
    size = (e.abs() * w.abs()).sum().double() * m * 2
    assert abs(float(left - right)) <= 4 * 6e-7 * float(size) + 1e-6 * float(x.abs().mul(w.abs()).sum())
