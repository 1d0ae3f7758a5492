"""Refusals of the history weight call that draft attention makes too (fake addresses, before any
device call)."""
import math

import pytest

from tree_forked_decision_b200 import flide

import test_decode_host as host
from test_decode_host import A, B, C, I, NUL, lib  # noqa: F401


@host.fake
@pytest.mark.parametrize("kw,code", [
    (dict(scale=-0.1), I), (dict(scale=math.nan), I), (dict(scale=math.inf), I), (dict(scale=-math.inf), I),
    (dict(idx=host._idx(T=1 << 28)), C), (dict(n_blocks=1 << 28), C), (dict(idx=host._idx(T=0)), flide.OK),
    (dict(idx=host._idx(T=0), scale=0.0), flide.OK),
])
def test_history_mass_refuses_what_draft_attention_refuses(lib, kw, code):  # noqa: F811
    a = dict(idx=host._idx(), n_blocks=4, scale=0.1)
    a.update(kw)
    ws = 1 << 40
    assert lib.flide_history_mass(A, A, A, A, a["n_blocks"], 16, A, 2, A, 2, a["idx"], 16, 4, 128, flide.BF16, NUL,
                                  a["scale"], A, B, NUL) == code
    assert lib.flide_draft_attn_paged(A, A, A, A, A, a["n_blocks"], 16, A, 2, A, 2, a["idx"], 16, 4, 128, flide.BF16,
                                      NUL, a["scale"], B, NUL, A, ws, NUL) == code
