"""The product's epilogue on every kernel that a call may take: the shape of its tiles is asserted with the library's
own rule, so that each case is what it is named."""
import pytest
import torch

from fp8_plan import ONE, ONE_SHARED, TWO, TWO_SHARED, Plan
from test_gpu_layer import Problem, no_errors_left, ops  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def plan_of(p, gated=False):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return Plan(sms, p.S, p.E, p.O // 2 if gated else p.O, p.depth, gated)


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


# counts, N, K, gated, the shape
SHAPES = [
    ([300], 1000, 256, False, ONE),
    ([100] * 100, 256, 256, False, TWO),
    ([1000], 4000, 528, False, TWO),
    ([2500, 0, 2600], 4096, 272, False, TWO),
    ([40], 1000, 1040, False, ONE_SHARED),
    ([5000], 2560, 272, True, TWO),
    ([128, 1, 129, 0] * 10, 1024, 256, True, TWO),
]


@pytest.mark.parametrize("gather", [0, 300])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32, "fp8"])
@pytest.mark.parametrize("counts,N,K,gated,shape", SHAPES)
def test_epilogue_of_every_shape(ops, counts, N, K, gated, shape, out, gather):  # noqa: F811
    p = Problem(ops, counts, N, K, seed=41, gather=gather)
    assert plan_of(p, gated).shape == shape
    F = p.O // 2 if gated else p.O
    out = ops.FP8 if out == "fp8" else out
    row_scale = torch.rand(p.S, **p.dev)
    for bias_dtype, dtype, act in ((torch.bfloat16, torch.float16, "silu"), (torch.float32, torch.bfloat16, None), (torch.float16, torch.float32, "gelu")):
        kw = dict(bias=torch.randn(p.E, p.O, **p.dev).to(bias_dtype), row_scale=row_scale, residual=torch.randn(p.S, F, **p.dev).to(dtype))
        p.check(p.run(activation=act, gated=gated, out=out, **kw), act=act, gated=gated, **kw)
    for kw in (dict(residual=torch.randn(p.S, F + 9, **p.dev).to(torch.bfloat16)[:, 3:3 + F]),       # rows off 16 bytes
               dict(residual=torch.randn(p.S, F, **p.dev).to(torch.bfloat16)), dict(row_scale=row_scale), dict(bias=torch.randn(p.E, p.O, **p.dev))):
        p.check(p.run(activation="relu", gated=gated, out=out, **kw), act="relu", gated=gated, **kw)
    if out != ops.FP8:                                # rows of the result off 16 bytes, the residual on them
        wide = torch.full((p.S, F + 9), 5.0, dtype=out, device="cuda")
        kw = dict(residual=torch.randn(p.S, F, **p.dev).to(torch.bfloat16))
        p.run(gated=gated, out=wide[:, 1:1 + F], **kw)
        p.check(wide[:, 1:1 + F], gated=gated, **kw)
        assert (wide[:, 0] == 5).all() and (wide[:, 1 + F:] == 5).all()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32, "fp8"])
@pytest.mark.parametrize("counts,N,K,shape", [([5000], 640, 4096, TWO), ([300], 256, 992, ONE), ([100] * 100, 256, 256, TWO), ([40], 1040, 1008, ONE_SHARED)])
def test_epilogue_of_transposed_products(ops, counts, N, K, shape, out):  # noqa: F811
    p = Problem(ops, counts, N, K, seed=43, transposed=True)
    assert plan_of(p).shape == shape
    kw = dict(bias=torch.randn(p.E, K, **p.dev), row_scale=torch.rand(p.S, **p.dev), residual=torch.randn(p.S, K, **p.dev).to(torch.bfloat16))
    p.check(p.run(activation="silu", out=ops.FP8 if out == "fp8" else out, **kw), act="silu", **kw)
