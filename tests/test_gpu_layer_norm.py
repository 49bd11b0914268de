"""The norm to FP8 rows where its squares leave float32's range: such rows are marked and done again."""
import pytest
import torch

from test_gpu_layer import check_quantized, gen, no_errors_left, ops, scales_of  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def normed(x, w, eps):
    """The normed rows in 64 bits, of sums x that were in float32 (or fewer bits) before."""
    x = x.double()
    return x / ((x * x).mean(1, keepdim=True) + eps).sqrt() * w.double()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [40, 64, 257, 1600, 5120, 5121, 20000])
def test_rows_whose_squares_overflow_or_underflow(ops, cols, dtype):  # noqa: F811
    g = gen(cols)
    size = torch.tensor([1e37, 1e25, 3e19, 1.0, 1e-25, 1e-37], device="cuda")[:, None]
    x = (torch.randn(6, cols, device="cuda", generator=g) * size).to(dtype)
    x[0, 0] = torch.finfo(dtype).max
    w = (1 + 0.3 * torch.randn(cols, device="cuda", generator=g)).to(dtype)
    for eps, r in ((0.0, None), (1e-6, torch.zeros_like(x))):
        q, _ = ops.rms_norm(x, w, ops.FP8, residual=r, eps=eps)
        y = normed(x, w, eps)
        check_quantized(q, y, y.abs() * 2.0 ** -20 + 2.0 ** -140)


@pytest.mark.parametrize("cols,off", [(64, 0), (64, 1), (640, 0), (4096, 0), (16400, 0)])
def test_many_rows_some_out_of_range(ops, cols, off):  # noqa: F811
    """Blocks that take several rows, the residual stream updated in place; a NaN weight of either sign marks nothing."""
    rows = 3000
    g = gen(cols + off)
    size = torch.ones(rows, 1, device="cuda")
    size[::5], size[3::7], size[2::11] = 1e30, 1e-30, 1e19
    x = (torch.randn(rows, cols, device="cuda", generator=g) * size).to(torch.bfloat16)
    r = (torch.randn(rows, cols + off, device="cuda", generator=g) * size).to(torch.bfloat16)[:, off:]
    w = (1 + 0.3 * torch.randn(cols, device="cuda", generator=g)).to(torch.bfloat16)
    r0, r1 = r.clone(), r.clone()
    q, total = ops.rms_norm(x, w, ops.FP8, residual=r, sum_out=r, eps=0.0)
    h = (x.double() + r0.double()).float().double()       # the sum of two bfloat16 values, rounded to float32
    y = normed(h, w, 0.0)
    check_quantized(q, y, y.abs() * 2.0 ** -20 + w.double().abs() * 2.0 ** -24)
    for sign in (-32768, 0):
        w2 = w.clone()
        w2.view(torch.int16)[0] = 0x7FC0 + sign
        r2 = r1.clone()
        q2, total2 = ops.rms_norm(x, w2, ops.FP8, residual=r2, sum_out=r2, eps=0.0)
        assert torch.equal(total2, total) and torch.equal(scales_of(q2)[:, 1:], scales_of(q)[:, 1:])
        assert scales_of(q2)[:, 0].isnan().all() and torch.equal(q2.codes[:, 128:], q.codes[:, 128:])


def test_one_huge_value(ops):  # noqa: F811
    x = torch.zeros(2, 64, device="cuda")
    x[0, 5], x[1, 3] = 3e37, 1e-30
    q, _ = ops.rms_norm(x, torch.ones(64, device="cuda"), ops.FP8, eps=1e-6)
    y = normed(x, torch.ones(64, device="cuda"), 1e-6)
    check_quantized(q, y, y.abs() * 2.0 ** -20 + 2.0 ** -140)
