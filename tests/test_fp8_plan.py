"""Which kernel a product of FP8 rows takes, by its sizes, on a GPU of 152 SMs.  No GPU needed."""
import random

import pytest

from fp8_plan import ONE, ONE_SHARED, PAIR, TWO, TWO_SHARED, Plan

SMS = 152


@pytest.mark.parametrize("slots,experts,F,depth,gated,rows,shape,split", [
    (1, 1, 2048, 5120, False, False, ONE_SHARED, 4),
    (64, 1, 5120, 5120, False, False, ONE_SHARED, 2),
    (16, 1, 2048, 5120, False, True, ONE_SHARED, 4),
    (1, 1, 2048, 256, False, False, ONE, 1),                # two blocks of depth are not shared
    (300, 1, 5120, 5120, False, False, ONE, 1),
    (300, 1, 1000, 256, False, False, ONE, 1),
    (10000, 100, 256, 1024, False, False, TWO, 1),
    (8191, 1, 5120, 5120, False, False, PAIR, 1),
    (8191, 1, 5120, 5120, False, True, TWO, 1),             # rows through an index take no pair
    (1000, 1, 4000, 528, False, False, PAIR, 1),
    (32768, 128, 2048, 2048, True, True, TWO, 1),
    (8191, 1, 4096, 5120, True, False, PAIR, 1),
])
def test_shapes(slots, experts, F, depth, gated, rows, shape, split):
    p = Plan(SMS, slots, experts, F, depth, gated, rows)
    assert (p.shape, p.split) == (shape, split) and p.stages >= 2


def sizes(n):
    rng = random.Random(5)
    for _ in range(n):
        gated = rng.random() < 0.5
        experts = 1 if rng.random() < 0.4 else int(2 ** rng.uniform(1, 13))
        yield dict(slots=int(2 ** rng.uniform(0, 16)), experts=experts, F=128 * rng.randint(1, 64) if gated else rng.randint(1, 8192),
                   depth=16 * rng.randint(1, 512), gated=gated, rows=rng.random() < 0.5)


def test_every_plan_can_be_launched():
    for c in sizes(20000):
        p = Plan(SMS, **c)
        # dynamic shared memory beside what the kernel has statically, a ring of two stages at least, tiles that hold every slot
        assert 2 <= p.stages <= 8 and p.smem <= 227 * 1024 - 10 * 1024, c
        assert p.split == 1 or (p.shape in (ONE_SHARED, TWO_SHARED) and p.split in (2, 4, 8)), c
        assert p.split > 1 or p.shape in (PAIR, ONE, TWO), c
        assert p.split == 1 or p.most_tiles * p.split <= 2 * SMS, c
        assert not (p.shape == PAIR and c["rows"]) and not (p.shape in (ONE, ONE_SHARED) and c["gated"]), c
        assert p.most_tiles * p.nt * p.tile_step >= c["slots"] * c["F"], c
