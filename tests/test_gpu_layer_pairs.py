"""Products on pairs of blocks, and the same through an index on blocks by themselves: what one warp hands to another
(rows, factors, partial sums) is there in every one of many calls, beside other work on the GPU and alone."""
import pytest
import torch

from fp8_plan import PAIR, TWO, Plan
from test_gpu_layer import Problem, no_errors_left, ops  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gather", [0, 700])
@pytest.mark.parametrize("counts,N,K,gated,transposed", [
    ([5000], 4000, 528, False, False), ([5000], 640, 4096, False, True), ([5000], 8192, 1040, True, False), ([2500, 0, 2600], 4096, 272, False, False),
    ([5000], 4000, 1040, False, False),
])
def test_pairs_repeat_themselves(ops, counts, N, K, gated, transposed, gather):  # noqa: F811
    p = Problem(ops, counts, N, K, seed=21, gather=gather, transposed=transposed)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert Plan(sms, p.S, p.E, p.O // 2 if gated else p.O, p.depth, gated, gather > 0).shape == (TWO if gather else PAIR)
    act = "silu" if gated else None
    want = p.run(out=torch.float32, activation=act, gated=gated)
    p.check(want, act=act, gated=gated)
    side = torch.cuda.Stream()
    a, b = torch.zeros(2, 1 << 26, dtype=torch.uint8, device="cuda")
    out, differ = torch.empty_like(want), torch.zeros((), dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    for i in range(200):
        if i % 2:                                     # beside copies that move the products' timing about
            with torch.cuda.stream(side):
                a[: (i * 77777) % (1 << 26)].copy_(b[: (i * 77777) % (1 << 26)])
        out.fill_(float("nan"))
        p.run(out=out, activation=act, gated=gated)
        differ += (out != want).sum()
    torch.cuda.synchronize()
    assert differ.item() == 0
