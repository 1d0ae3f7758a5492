"""Eviction of histories longer than the rows that a block's selection holds at a time."""
import pytest
import torch

import test_gpu_evict as short

pytestmark = pytest.mark.gpu

SHAPES = [  # lengths, budget, sinks, recent, block rows, (Hkv, d), type
    ([16384, 16385], 16300, 3, 5000, 16, (1, 8), torch.bfloat16),
    ([33000, 16383, 700], 20001, 4, 64, 48, (2, 8), torch.uint8),
    ([50001], 16390, 0, 1, 7, (1, 4), torch.float32),          # slots that start at odd places
    ([40003, 39999], 39998, 20000, 19000, 11, (1, 8), torch.bfloat16),
    ([70000], 35000, 17000, 17999, 128, (1, 8), torch.bfloat16),
]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"{s[0][0]}to{s[1]}" for s in SHAPES])
def test_evict_many_chunks(shape, kind, in_place):
    short.test_evict(shape, kind, in_place)
