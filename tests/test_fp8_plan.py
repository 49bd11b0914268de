"""Which kernel a product of FP8 rows takes, by its sizes, on a GPU of 152 SMs.  No GPU needed."""
import random

import pytest

from fp8_plan import ONE, ONE_SHARED, TWO, TWO_SHARED, Plan

SMS = 152


@pytest.mark.parametrize("slots,experts,F,depth,gated,shape,split", [
    (1, 1, 2048, 5120, False, ONE_SHARED, 4),
    (64, 1, 5120, 5120, False, ONE_SHARED, 2),
    (1, 1, 2048, 256, False, ONE, 1),                # two blocks of depth are not shared
    (300, 1, 5120, 5120, False, ONE, 1),
    (300, 1, 1000, 256, False, ONE, 1),
    (512, 1, 5120, 5120, False, TWO, 1),
    (8191, 1, 5120, 5120, False, TWO, 1),
    (10000, 100, 256, 1024, False, TWO, 1),
    (32768, 128, 2048, 2048, True, TWO, 1),
    (8191, 1, 4096, 5120, True, TWO, 1),
])
def test_shapes(slots, experts, F, depth, gated, shape, split):
    p = Plan(SMS, slots, experts, F, depth, gated)
    assert (p.shape, p.split) == (shape, split) and p.stages >= 2


def sizes(n):
    rng = random.Random(5)
    for _ in range(n):
        gated = rng.random() < 0.5
        experts = 1 if rng.random() < 0.4 else int(2 ** rng.uniform(1, 13))
        yield dict(slots=int(2 ** rng.uniform(0, 16)), experts=experts, F=128 * rng.randint(1, 64) if gated else rng.randint(1, 8192),
                   depth=16 * rng.randint(1, 512), gated=gated)


def test_every_plan_can_be_launched():
    for c in sizes(20000):
        p = Plan(SMS, **c)
        # dynamic shared memory beside what the kernel has statically, a ring of two stages at least, tiles that hold every slot
        assert 2 <= p.stages <= 8 and p.smem <= 227 * 1024 - 10 * 1024, c
        assert (p.split == 1 and p.shape in (ONE, TWO)) or (p.split in (2, 4, 8) and p.shape in (ONE_SHARED, TWO_SHARED)), c
        assert p.split == 1 or p.most_tiles * p.split <= 2 * SMS, c
        assert not (p.shape in (ONE, ONE_SHARED) and c["gated"]), c
        assert p.most_tiles * p.nt * p.tile_step >= c["slots"] * c["F"], c


@pytest.mark.parametrize("slots,experts,F,depth,split", [
    (1, 1, 2048, 5120, 4), (32, 1, 2048, 5120, 4), (128, 1, 2048, 5120, 2), (1, 1, 512, 2048, 8), (64, 1, 512, 1600, 4),
    (8, 128, 512, 1600, 2), (2, 6000, 128, 1024, 4), (1, 1, 128, 512, 2),
])
def test_gated_products_of_few_slots_share_their_depth(slots, experts, F, depth, split):
    p = Plan(SMS, slots, experts, F, depth, True)
    assert (p.shape, p.split) == (TWO_SHARED, split)


def test_prefixes_of_many_experts_leave_no_room_to_share_a_gated_products_depth():
    # 8 bytes an expert beside 64 KB of sums and two stages of 48 KB
    assert Plan(SMS, 2, 6000, 128, 1024, True).split == 4
    p = Plan(SMS, 2, 8192, 128, 1024, True)
    assert p.split == 1 and p.shape == TWO and p.stages >= 2
    assert Plan(SMS, 2, 8192, 128, 1024).split == 4          # half the sums: there is room


def test_two_blocks_share_a_gated_product_where_it_pays():
    # (the kernels' times are beside the rule)
    for slots, experts, F, depth, split in ((64, 1, 4096, 2048, 1), (32, 1, 4096, 2048, 2), (1, 1, 8192, 2048, 2), (256, 1, 2048, 5120, 2), (256, 1, 2048, 1024, 1),
                                            (64, 1, 512, 1024, 4), (128, 8, 512, 1600, 2), (1024, 8, 256, 1600, 1)):
        assert Plan(SMS, slots, experts, F, depth, True).split == split, (slots, experts, F, depth)


def test_few_tiles_share_their_depth_gated_or_not():
    seen = set()
    for c in sizes(20000):
        p = Plan(SMS, **c)
        seen.add(p.shape)
        slot_tiles = -(-c["slots"] // 64) if c["experts"] == 1 else min(c["experts"], c["slots"]) + c["slots"] // 64
        few = -(-c["F"] // 128) * slot_tiles
        if few * 2 <= SMS and c["depth"] > 3 * 128 and c["experts"] < 5000:
            deep = few * 4 <= SMS // 2 and c["depth"] > 7 * 128
            assert p.split > 1 or (c["gated"] and not deep), c
            assert p.split >= 4 or not deep, c
    assert seen == {ONE, TWO, ONE_SHARED, TWO_SHARED}         # every kernel is some product's
