"""The operators of csf_layer.h against plain 64-bit definitions: FP8 rows,
products with a scale for each block of 128, tokens to slots and back, and the
gradients of that way and of the router."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}     # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


@pytest.fixture(scope="module")
def ops():
    from lossless_nvfp4_scale_gb300 import build
    build.ensure_built()
    from lossless_nvfp4_scale_gb300 import ops as mod
    return mod


@pytest.fixture(autouse=True)
def no_errors_left(ops):
    yield
    assert ops.errors() == 0


def up(n, m):
    return -(-n // m) * m


def blocks(n):
    return -(-n // 128)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def scales_of(q):
    return q.scales.view(torch.float32)[:, :blocks(q.cols)]


def values(q):
    """FP8 rows as the values they stand for, in 64 bits."""
    v = q.codes.view(torch.float8_e4m3fn)[:, :q.cols].double()
    return v * scales_of(q).double().repeat_interleave(128, 1)[:, :q.cols]


def quantized(y):
    """FP8 codes and scales of rows in 64 bits by the definition: codes [rows, cols], scales float32."""
    y = torch.nn.functional.pad(y, (0, up(y.shape[1], 128) - y.shape[1]))
    v = y.view(y.shape[0], -1, 128)
    scale = (v.abs().amax(2).float() / 448).clamp(min=2.0 ** -126)
    return v / scale.double()[..., None], scale


def check_quantized(q, y, slack=None):
    """FP8 rows against 64-bit values y [rows, cols] that were in float32
    before (slack None: exactly y), or within slack [rows, cols] of y.

    A scale is m / 448 rounded, m the block's largest magnitude: within 2^-24
    and m's own error / 448 of it.  A code is off by half a step of E4M3
    (2^-4 relative, 2^-10 at least), plus what the value and scale are off."""
    rows, cols = y.shape
    assert (q.codes[:, cols:] == 0).all()
    got_scale = scales_of(q).double()
    assert (q.scales.view(torch.float32)[:, blocks(cols):] == 0).all()
    pad = (0, up(cols, 128) - cols)
    v = torch.nn.functional.pad(y, pad).view(rows, -1, 128)
    e = torch.nn.functional.pad(slack if slack is not None else torch.zeros_like(y), pad).view(rows, -1, 128)
    m = v.abs().amax(2)
    want = (m / 448).clamp(min=2.0 ** -126)
    assert ((got_scale - want).abs() <= want * 2.0 ** -23 + e.amax(2) / 448).all()
    if slack is None:
        exact, scale = quantized(y)
        assert torch.equal(scale.double(), got_scale)
    code = torch.nn.functional.pad(q.codes.view(torch.float8_e4m3fn)[:, :cols].double(), pad).view(rows, -1, 128)
    ratio = v / got_scale[..., None]
    off = (code - ratio).abs()
    # a quotient next to the middle of two codes may have been rounded in 32 bits before
    assert (off <= torch.maximum(ratio.abs() * 2.0 ** -4, torch.full_like(ratio, 2.0 ** -10)) * (1 + 2.0 ** -20)
            + e / got_scale[..., None] * 1.01).all()


def close(got, want, slack):
    """Within `slack` and a rounding to got's type of want, NaN alike."""
    w = want.double()
    bound = slack + w.abs() * STEP[got.dtype] * (1 + 2.0 ** -10) + TINY[got.dtype]
    off = (got.double() - w).abs()
    assert (off <= bound).all(), (off / bound).max()


# ---- the product ---------------------------------------------------------------------------------------------------

def act64(v, name):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v.clamp(min=0) if name == "relu" else v


class Problem:
    def __init__(self, ops, counts, N, K, seed=0, gather=0, tail=0, transposed=False):
        g = gen(seed)
        dev = dict(device="cuda", generator=g)
        self.ops, self.N, self.K, self.E, self.transposed = ops, N, K, len(counts), transposed
        self.used, self.S = sum(counts), sum(counts) + tail
        self.T = gather or max(self.S, 1)
        self.depth, self.O = (N, K) if transposed else (K, N)
        codes = (torch.randn(self.T, up(self.depth, 32), **dev) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        codes[:, self.depth:] = 0
        sc = torch.zeros(self.T, up(4 * blocks(self.depth), 16) // 4, device="cuda")
        sc[:, :blocks(self.depth)] = torch.rand(self.T, blocks(self.depth), **dev) + 0.01
        self.x = ops.Quantized(ops.FP8, codes.view(torch.uint8), sc.view(torch.uint8), self.depth)
        self.w = (torch.randn(self.E, N, K, **dev) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        self.ws = (torch.rand(self.E, blocks(N), blocks(K), **dev) + 0.01) / (1e4 * self.depth ** 0.5)
        self.start = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
        self.rows = torch.randint(0, self.T, (self.S,), dtype=torch.int32, **dev) if gather else None
        self.expert = torch.repeat_interleave(torch.arange(self.E, device="cuda"), self.start.diff().long())
        self.dev = dev

    def sums(self):
        """The used slots' products in 64 bits, and the sums of their terms' magnitudes."""
        x = values(self.x)[self.rows.long() if self.rows is not None else slice(0, self.S)][:self.used]
        y = torch.zeros(self.used, self.O, dtype=torch.float64, device="cuda")
        size = torch.zeros_like(y)
        for e in range(self.E):
            m = self.expert == e
            if m.any():
                s = self.ws[e].double().repeat_interleave(128, 0)[:self.N].repeat_interleave(128, 1)[:, :self.K]
                w = self.w[e].double() * s
                w = w if self.transposed else w.T
                y[m], size[m] = x[m] @ w, x[m].abs() @ w.abs()
        return y, size

    def check(self, out, bias=None, act=None, gated=False, row_scale=None, residual=None):
        y, size = self.sums()
        # sums of `depth` products in 32 bits, a matrix step of 32 at a time; a factor of two roundings
        slack = size * (self.depth / 32 + 4) * 2.0 ** -23
        if bias is not None:
            y = y + bias.double()[self.expert]
            slack = slack + y.abs() * 2.0 ** -24
        slope = {None: 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13}[act]        # the steepest that the functions get
        # their own error is 2^-20 of the value, GELU's 2^-21 |z| more, z up to 1.6 (|v| + 0.045 |v|^3)
        own = {None: 0.0, "relu": 0.0, "silu": 2.0 ** -20}.get(act)
        v = y[:, :self.O // 2] if gated else y
        e = slack[:, :self.O // 2] if gated else slack
        a = act64(v, act)
        ea = e * slope + a.abs() * (own if own is not None else 2.0 ** -20 + 2.0 ** -21 * 1.6 * (v.abs() + 0.045 * v.abs() ** 3))
        if gated:
            u, eu = y[:, self.O // 2:], slack[:, self.O // 2:]
            y, slack = a * u, ea * u.abs() + a.abs() * eu + ea * eu + (a * u).abs() * 2.0 ** -24
        else:
            y, slack = a, ea
        if row_scale is not None:
            r = row_scale.double()[:self.used, None]
            y, slack = y * r, slack * r.abs() + (y * r).abs() * 2.0 ** -24
        if residual is not None:
            y = y + residual.double()[:self.used]
            slack = slack + y.abs() * 2.0 ** -24
        if isinstance(out, self.ops.Quantized):
            check_quantized(self.ops.Quantized(out.kind, out.codes[:self.used], out.scales[:self.used], out.cols), y, slack)
        else:
            close(out[:self.used], y, slack)

    def run(self, **kw):
        return self.ops.fp8_matmul(self.x, self.w, self.ws, expert_start=self.start if self.E > 1 or self.used < self.S else None,
                                   rows=self.rows, transposed=self.transposed, **kw)


@pytest.mark.parametrize("counts,N,K,gather", [
    ([1], 128, 128, 0), ([1], 2048, 5120, 0), ([3], 200, 1600, 0), ([17], 40, 16, 5), ([64], 1000, 2048, 0), ([65], 384, 144, 0),
    ([128], 256, 256, 0), ([129], 256, 256, 0), ([300], 300, 400, 0), ([257], 1, 640, 70), ([1000], 4000, 528, 0),
    ([2, 0, 5, 0, 1], 300, 1040, 7), ([40, 0, 131, 300], 260, 336, 100), ([200] * 9, 520, 656, 0), ([513, 0, 1, 255], 128, 4400, 33),
])
def test_product(ops, counts, N, K, gather):
    p = Problem(ops, counts, N, K, seed=N + K, gather=gather)
    p.check(p.run(out=torch.float32))


@pytest.mark.parametrize("counts,N,K,gather", [
    ([1], 128, 128, 0), ([5], 2048, 1600, 0), ([64], 400, 1008, 9), ([130], 336, 272, 0), ([600], 1040, 4000, 0), ([300, 0, 7, 220], 240, 640, 50),
])
def test_transposed_product(ops, counts, N, K, gather):
    p = Problem(ops, counts, N, K, seed=N + K, gather=gather, transposed=True)
    bias = torch.randn(p.E, K, **p.dev)
    p.check(p.run(out=torch.float32, bias=bias), bias=bias)


@pytest.mark.parametrize("counts", [[7], [150], [3, 0, 40, 131], [300, 0, 260]])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32, "fp8"])
@pytest.mark.parametrize("act,gated", [(None, False), ("relu", False), ("gelu", False), ("silu", False), ("silu", True), ("gelu", True)])
def test_epilogue(ops, counts, act, gated, out):
    p = Problem(ops, counts, 512 if gated else 200, 400, seed=3, gather=50)
    F = p.O // 2 if gated else p.O
    kw = dict(bias=torch.randn(p.E, p.O, **p.dev).to(torch.bfloat16), row_scale=torch.rand(p.S, **p.dev),
              residual=torch.randn(p.S, F, **p.dev).to(torch.float16))
    p.check(p.run(activation=act, gated=gated, out=ops.FP8 if out == "fp8" else out, **kw), act=act, gated=gated, **kw)
    p.check(p.run(activation=act, gated=gated, out=ops.FP8 if out == "fp8" else out), act=act, gated=gated)


@pytest.mark.parametrize("N", [1, 31, 33, 128, 129, 250, 1000])
@pytest.mark.parametrize("counts", [[5], [70, 90], [300]])
def test_ragged_quantized_outputs(ops, N, counts):
    p = Problem(ops, counts, N, 256, seed=4)
    p.check(p.run(out=ops.FP8))
