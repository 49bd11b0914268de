"""The product's epilogue on every kernel that a call may take: the shape of its tiles is asserted with the library's
own rule, so that each case is what it is named."""
import pytest
import torch

from fp8_plan import TWO_SHARED, Plan
from test_gpu_layer import Problem, no_errors_left, ops  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def plan_of(p, gated=False):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return Plan(sms, p.S, p.E, p.O // 2 if gated else p.O, p.depth, gated, p.rows is not None)


@pytest.mark.parametrize("gather", [0, 40])
@pytest.mark.parametrize("counts,N,K,split", [([1], 4096, 5120, 4), ([64], 1024, 2048, 8), ([30], 256, 528, 2), ([5, 0, 70], 512, 1040, 4)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32, "fp8"])
def test_gated_products_that_share_their_depth(ops, counts, N, K, split, gather, out):  # noqa: F811
    p = Problem(ops, counts, N, K, seed=31, gather=gather)
    plan = plan_of(p, True)
    assert (plan.shape, plan.split) == (TWO_SHARED, split)
    kw = dict(bias=torch.randn(p.E, p.O, **p.dev).to(torch.bfloat16), row_scale=torch.rand(p.S, **p.dev),
              residual=torch.randn(p.S, N // 2, **p.dev).to(torch.float16))
    out = ops.FP8 if out == "fp8" else out
    for act in ("silu", "gelu"):
        p.check(p.run(activation=act, gated=True, out=out, **kw), act=act, gated=True, **kw)
    first = p.run(activation="silu", gated=True, out=out)
    p.check(first, act="silu", gated=True)
    for _ in range(3):                                # the order of the blocks' sums does not change
        again = p.run(activation="silu", gated=True, out=out)
        assert torch.equal(again.codes, first.codes) if isinstance(first, ops.Quantized) else torch.equal(again, first)


def test_gated_product_beside_the_prefix_of_many_experts(ops):  # noqa: F811
    """6000 experts' prefix leaves room for clusters that share the depth, 8192 experts' does not."""
    for E, split in ((6000, 4), (8192, 1)):
        p = Problem(ops, [2], 256, 1024, seed=10)
        assert Plan(152, 2, E, 128, 1024, True).split == split
        w, ws = p.w.view(torch.uint8).expand(E, -1, -1).contiguous(), p.ws.expand(E, -1, -1).contiguous()
        start = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        start[E:] = 2
        for out in (torch.float32, ops.FP8):
            p.check(ops.fp8_matmul(p.x, w, ws, expert_start=start, out=out, gated=True, activation="silu"), act="silu", gated=True)
