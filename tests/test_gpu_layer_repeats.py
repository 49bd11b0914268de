"""Products on every shape of tile: what one warp hands to another (rows, factors, partial sums), and one block of a
cluster to the next, is there in every one of many calls, beside other work on the GPU and alone."""
import pytest
import torch

from fp8_plan import ONE, ONE_SHARED, TWO, TWO_SHARED
from test_gpu_layer import Problem, no_errors_left, ops  # noqa: F401  (fixtures)
from test_gpu_layer_shapes import plan_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gather", [0, 700])
@pytest.mark.parametrize("counts,N,K,gated,transposed,shape", [
    ([5000], 4000, 528, False, False, TWO), ([5000], 640, 4096, False, True, TWO), ([5000], 8192, 1040, True, False, TWO),
    ([300], 1000, 256, False, False, ONE), ([3000, 0, 2900], 300, 272, False, False, ONE),
    ([64], 1000, 2048, False, False, ONE_SHARED), ([60], 1024, 2048, True, False, TWO_SHARED),
])
def test_products_repeat_themselves(ops, counts, N, K, gated, transposed, shape, gather):  # noqa: F811
    p = Problem(ops, counts, N, K, seed=21, gather=gather, transposed=transposed)
    assert plan_of(p, gated).shape == shape
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
