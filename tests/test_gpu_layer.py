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
    scale = (v.abs().amax(2) / 448).float().clamp(min=2.0 ** -126)      # (in 32 bits torch multiplies by 1 / 448)
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


@pytest.mark.parametrize("counts,N,K,gated,transposed", [
    ([900], 5120, 256, False, False),                # a pair of blocks a tile
    ([1200], 640, 4096, False, True),
    ([700], 2560, 256, True, False),
    ([130] * 12, 2560, 256, False, False),           # 256 columns a block
    ([100] * 16, 640, 2560, False, True),
    ([100] * 40, 256, 2048, False, True),
    ([128, 1, 129, 0] * 10, 1024, 256, True, False),
    ([140] * 3, 256, 384, False, False),             # 128 columns a block
])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32, "fp8"])
def test_tile_shapes(ops, counts, N, K, gated, transposed, out):
    for gather in (0, 300):
        p = Problem(ops, counts, N, K, seed=8, gather=gather, transposed=transposed)
        act = "silu" if gated else None
        p.check(p.run(activation=act, gated=gated, out=ops.FP8 if out == "fp8" else out), act=act, gated=gated)


def test_slots_past_the_last_expert_stay(ops):
    for counts, N in (([3, 9], 256), ([300, 300], 2560)):
        p = Problem(ops, counts, N, 256, seed=2, gather=20, tail=7)
        out = torch.full((p.S, N), 7.0, device="cuda")
        p.run(out=out)
        p.check(out)
        assert (out[p.used:] == 7).all()
        q = ops.empty_quantized(ops.FP8, p.S, N)
        q.codes.fill_(9), q.scales.fill_(9)
        p.run(out=q)
        p.check(q)
        assert (q.codes[p.used:] == 9).all() and (q.scales[p.used:] == 9).all()


def test_strided_and_unaligned_operands(ops):
    p = Problem(ops, [70, 200], 328, 400, seed=5)
    wide = torch.zeros(p.S, 1024, dtype=torch.uint8, device="cuda")
    wide[:, 64:64 + p.x.codes.shape[1]] = p.x.codes
    sc = torch.zeros(p.S, 96, dtype=torch.uint8, device="cuda")
    sc[:, 32:32 + p.x.scales.shape[1]] = p.x.scales
    p.x = ops.Quantized(ops.FP8, wide[:, 64:64 + p.x.codes.shape[1]], sc[:, 32:32 + p.x.scales.shape[1]], 400)
    for dtype in DTYPES:
        out = torch.full((p.S, 341), 5.0, dtype=dtype, device="cuda")
        res = torch.randn(p.S, 345, **p.dev).to(dtype)
        bias = torch.randn(2 * 328 + 1, **p.dev).to(dtype)[1:].view(2, 328)
        p.run(out=out[:, 1:329], residual=res[:, 3:331], bias=bias)
        p.check(out[:, 1:329], residual=res[:, 3:331], bias=bias)
        assert (out[:, 0] == 5).all() and (out[:, 329:] == 5).all()


def test_bad_rows_and_expert_starts_are_reported(ops):
    for counts, N in (([5], 200), ([200, 300], 2560), ([300], 5120)):
        p = Problem(ops, counts, N, 256, seed=6, gather=30)
        p.rows[2], p.rows[4] = 30, -5
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = p.run(out=torch.float32, error_word=word)
        assert word.item() != 0
        p.rows[2] = p.rows[4] = 0                     # what they stand for
        p.check(out)
    p = Problem(ops, [5, 6], 200, 256, seed=6)
    for start in ([0, 7, 5], [0, 5, 12], [-1, 5, 11]):
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((11, 200), 3.0, device="cuda")
        ops.fp8_matmul(p.x, p.w, p.ws, expert_start=torch.tensor(start, dtype=torch.int32, device="cuda"), out=out, error_word=word)
        assert word.item() != 0 and (out == 3).all()


def test_nan_and_infinite_scales_stay_with_their_rows(ops):
    p = Problem(ops, [9, 140], 300, 640, seed=7)
    p.x.codes[3, 5] = 0x7F                            # a NaN code
    sc = p.x.scales.view(torch.float32)
    sc[20, 1], sc[140, 2] = math.nan, math.inf
    p.x.codes[140, 256:384] = 0x38                    # ones: no 0 times infinity
    out = p.run(out=torch.float32)
    bad = torch.zeros(149, dtype=torch.bool, device="cuda")
    bad[[3, 20, 140]] = True
    assert (~out[bad].isfinite()).all() and out[~bad].isfinite().all()
    q = p.run(out=ops.FP8)
    assert scales_of(q)[bad].isnan().all() and scales_of(q)[~bad].isfinite().all()


def test_product_is_deterministic_and_captured(ops):
    """Replays of a captured call, and calls on two streams at once, give the eager call's bits."""
    for counts, N, K in (([1], 2048, 2560), ([40, 300], 512, 640), ([700], 5120, 512)):
        p = Problem(ops, counts, N, K, seed=9, gather=25)
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        want = p.run(error_word=word)
        out = torch.zeros_like(want)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p.run(out=out, error_word=word)
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        ya, yb = p.run(stream=a, error_word=word), p.run(stream=b, error_word=word)
        torch.cuda.synchronize()
        assert torch.equal(ya, want) and torch.equal(yb, want) and word.item() == 0


def test_one_expert_of_8192(ops):
    """The prefix over many experts, most of them without slots."""
    E = 8192
    p = Problem(ops, [3], 128, 128, seed=10)
    w = p.w.view(torch.uint8).expand(E, -1, -1).contiguous()
    ws = p.ws.expand(E, -1, -1).contiguous()
    start = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    start[5001:] = 3
    p.check(ops.fp8_matmul(p.x, w, ws, expert_start=start, out=torch.float32))


def test_gated_product_of_few_slots_on_8192_experts(ops):
    """Prefixes of many experts leave no room for clusters that share the depth."""
    E = 8192
    p = Problem(ops, [2], 256, 1024, seed=10)
    w, ws = p.w.view(torch.uint8).expand(E, -1, -1).contiguous(), p.ws.expand(E, -1, -1).contiguous()
    start = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    start[8192:] = 2
    for out in (torch.float32, ops.FP8):
        p.check(ops.fp8_matmul(p.x, w, ws, expert_start=start, out=out, gated=True, activation="silu"), act="silu", gated=True)


def test_many_choices_a_token(ops):
    T, k, H = 5, 70, 200
    g = gen(6)
    slots = torch.randperm(T * k, device="cuda", generator=g).int().view(T, k)
    slots[1, 3:60], slots[4] = -1, -1
    y, w = torch.randn(T * k, H, device="cuda", generator=g), torch.randn(T, k, device="cuda", generator=g)
    go = torch.randn(T, H, device="cuda", generator=g)
    want = combine64(y.double(), slots, w.double(), None)
    close(ops.combine(y, slots, w), want, combine64(y.double().abs(), slots, w.double().abs(), None) * k * 2.0 ** -24)
    dy, dw = ops.combine_grad(go, y, slots, w)
    on = slots >= 0
    rows = y.double()[slots.clamp(min=0).long()]
    want = torch.where(on, (go.double()[:, None] * rows).sum(2), 0)
    close(dw, want, (go.double().abs()[:, None] * rows.abs()).sum(2) * 24 * 2.0 ** -24)
    want = (w.double()[..., None] * go.double()[:, None])[on]
    close(dy[slots[on].long()], want, want.abs() * 2.0 ** -24)
    out = ops.dispatch(go, slots)
    assert torch.equal(out[slots[on].long()], go[:, None].expand(-1, k, -1)[on])


def test_weights_past_32_bit_offsets(ops):
    E, N, K = 3, 40000, 20000                         # 2.4e9 bytes of weights
    x = ops.quantize(torch.randn(5, K, device="cuda"), ops.FP8)
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    w[2, N - 300:] = torch.randint(0x20, 0x40, (300, K), dtype=torch.uint8, device="cuda")
    ws = torch.rand(E, blocks(N), blocks(K), device="cuda")
    start = torch.tensor([0, 0, 0, 5], dtype=torch.int32, device="cuda")
    y = ops.fp8_matmul(x, w, ws, expert_start=start, out=torch.float32)
    s = ws[2].double().repeat_interleave(128, 0)[N - 300:N].repeat_interleave(128, 1)[:, :K]
    wv = w[2, N - 300:].view(torch.float8_e4m3fn).double() * s
    xv = values(x)
    close(y[:, N - 300:], xv @ wv.T, (xv.abs() @ wv.T.abs()) * (K / 32 + 4) * 2.0 ** -23)
    assert (y[:, :N - 300] == 0).all()


# ---- FP8 rows ------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (7, 33), (2, 128), (5, 129), (33, 1001), (300, 1600), (9, 5120), (2, 20000)])
def test_quantize(ops, rows, cols, dtype):
    g = gen(rows + cols)
    x = (torch.randn(rows, cols, device="cuda", generator=g) * torch.rand(rows, 1, device="cuda", generator=g)).to(dtype)
    check_quantized(ops.quantize(x, ops.FP8), x.double())
    for kind in (ops.NVFP4, ops.MXFP8):               # as the norm makes them, of values that it leaves alone
        q = ops.quantize(x, kind)
        wide = torch.zeros(rows, up(cols, 8) + 8, dtype=dtype, device="cuda")
        wide[:, 1:1 + cols] = x
        q2 = ops.quantize(wide[:, 1:1 + cols], kind)  # off 16 bytes
        assert torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales)


@pytest.mark.parametrize("kind", [0, 1])
def test_quantize_of_the_other_kinds_is_the_norms(ops, kind):
    """Rows of ones and minus ones have mean square 1: the norm by a weight is a product with it, exactly."""
    g = gen(4)
    w = (torch.randn(640, device="cuda", generator=g) * 3).to(torch.bfloat16)
    x = torch.where(torch.rand(50, 640, device="cuda", generator=g) < 0.5, -1.0, 1.0).to(torch.bfloat16)
    ts = torch.tensor([0.01], device="cuda") if kind == ops.NVFP4 else None
    n, _ = ops.rms_norm(x, w, kind, eps=0.0, tensor_scale=ts)
    q = ops.quantize(x * w, kind, tensor_scale=ts)
    assert torch.equal(n.codes, q.codes) and torch.equal(n.scales, q.scales)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 128), (5, 200), (40, 1600), (3, 4097), (2, 20000)])
def test_norm_to_fp8(ops, rows, cols, dtype):
    g = gen(cols)
    x = torch.randn(rows, cols, device="cuda", generator=g).to(dtype)
    r = torch.randn(rows, cols, device="cuda", generator=g).to(dtype)
    w = (1 + 0.2 * torch.randn(cols, device="cuda", generator=g)).to(dtype)
    q, total = ops.rms_norm(x, w, ops.FP8, residual=r, eps=1e-5)
    h = x.double() + r.double()
    y = h / ((h * h).mean(1, keepdim=True) + 1e-5).sqrt() * w.double()
    # h's rounding, the sum's (its terms' share halves), the root's 2^-22 and three products
    check_quantized(q, y, y.abs() * 2.0 ** -20 + w.double().abs() * 2.0 ** -24)
    close(total, h, 0)


def test_extreme_values_quantize(ops):
    x = torch.zeros(8, 256, device="cuda")
    x[1, 0], x[1, 200] = 3e38, -1e-3
    x[2] = 1e-42                                      # below the least scale's codes
    x[3, :128] = 2.0 ** -126
    x[4, 5], x[5, 6], x[6, 130] = math.inf, math.nan, -math.inf
    x[7] = torch.linspace(-448, 448, 256)
    q = ops.quantize(x, ops.FP8)
    s = scales_of(q)
    assert s[4, 0].isnan() and s[5, 0].isnan() and s[6, 1].isnan()
    assert s[[4, 5], 1].isfinite().all() and s[6, 0].isfinite()
    keep = torch.tensor([0, 1, 2, 3, 7], device="cuda")
    check_quantized(ops.Quantized(ops.FP8, q.codes[keep], q.scales[keep], 256), x[keep].double())
    assert (s[0] == 2.0 ** -126).all() and (q.codes[0] == 0).all()


# ---- to slots and back ---------------------------------------------------------------------------------------------

def routes(ops, T, k, E, seed, masked):
    g = gen(seed)
    logits = torch.randn(T, E, device="cuda", generator=g)
    if masked:
        logits[torch.rand(T, E, device="cuda", generator=g) < 0.5] = -math.inf
        logits[::3, 1:] = -math.inf
        logits[1::4] = -math.inf
    return ops.route(logits, k), logits


CASES = [(1, 1, 1, False), (1, 5120, 8, False), (3, 33, 2, True), (50, 1001, 6, True), (700, 128, 8, False), (2500, 72, 3, True), (5, 8000, 32, False),
         (40, 264, 1, True)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,k,masked", CASES)
def test_dispatch_and_its_gradient(ops, T, H, k, masked, dtype):
    r, _ = routes(ops, T, k, max(40, k), T + H, masked)
    x = torch.randn(T, H, device="cuda", generator=gen(H)).to(dtype)
    out = torch.full((T * k, H), 3.0, dtype=dtype, device="cuda")
    ops.dispatch(x, r.slots, out=out)
    used = (r.rows >= 0).nonzero().view(-1)
    assert torch.equal(out[used], x[r.rows[used].long()]) and (out[r.rows < 0] == 3).all()
    for other in DTYPES:
        assert torch.equal(ops.dispatch(x, r.slots, out=other)[used], x[r.rows[used].long()].to(other))
    for kind in (ops.FP8, ops.NVFP4, ops.MXFP8):
        q, one = ops.empty_quantized(kind, T * k, H), ops.quantize(x, kind)
        q.codes.fill_(7), q.scales.fill_(7)
        ops.dispatch(x, r.slots, out=q)
        assert torch.equal(q.codes[used], one.codes[r.rows[used].long()]) and torch.equal(q.scales[used], one.scales[r.rows[used].long()])
        assert (q.codes[r.rows < 0] == 7).all() and (q.scales[r.rows < 0] == 7).all()
    # <g, dispatch(x)> is linear in x: its gradient is each token's rows of g, summed
    g = torch.randn(T * k, H, device="cuda", generator=gen(1)).to(dtype)
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    want.index_add_(0, r.rows[used].long(), g[used].double())
    size.index_add_(0, r.rows[used].long(), g[used].double().abs())
    close(ops.dispatch_grad(g, r.slots), want, size * k * 2.0 ** -24)


def combine64(y, slots, weights, residual):
    rows = torch.where((slots >= 0)[..., None], y[slots.clamp(min=0).long()], torch.zeros((), dtype=y.dtype, device=y.device))
    out = (weights[..., None] * rows).sum(1)
    return out if residual is None else out + residual


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,H,k,masked", CASES)
def test_combine_and_its_gradient(ops, T, H, k, masked, dtype):
    r, _ = routes(ops, T, k, max(40, k), T + H, masked)
    g = gen(T)
    y = torch.randn(T * k, H, device="cuda", generator=g).to(dtype)
    y[r.rows < 0] = math.nan                          # what no choice names is not read
    w = torch.rand(T, k, device="cuda", generator=g)
    w[r.slots < 0] = math.nan                         # nor the weights of choices that fell away
    res = torch.randn(T, H, device="cuda", generator=g).to(torch.float16)
    w64 = torch.nan_to_num(w.double())
    y64 = y.double()
    want = combine64(y64, r.slots, w64, res.double())
    slack = combine64(y64.abs(), r.slots, w64, res.double().abs()) * (k + 2) * 2.0 ** -24
    close(ops.combine(y, r.slots, w, residual=res, out=torch.float32), want, slack)
    close(ops.combine(y, r.slots, w, residual=res), want, slack)
    close(ops.combine(y, r.slots, out=torch.float32), combine64(y64, r.slots, torch.ones_like(w64), None),
          combine64(y64.abs(), r.slots, torch.ones_like(w64), None) * k * 2.0 ** -24)
    same = res.clone()                                # the residual stream in place
    ops.combine(y, r.slots, w, residual=same, out=same)
    close(same, want, slack)
    # gradients: the formula by autograd in 64 bits
    go = torch.randn(T, H, device="cuda", generator=g).to(dtype)
    yl, wl = torch.nan_to_num(y64).requires_grad_(), w64.clone().requires_grad_()
    combine64(yl, r.slots, wl, None).backward(go.double())
    dy = torch.full((T * k, H), 3.0, dtype=dtype, device="cuda")
    _, dw = ops.combine_grad(go, y, r.slots, w, out=dy)
    used = r.rows >= 0
    close(dy[used], yl.grad[used], yl.grad[used].abs() * 2.0 ** -24)
    assert (dy[~used] == 3).all()
    size = (go.double().abs()[:, None] * torch.nan_to_num(y64)[r.slots.clamp(min=0).long()].abs()).sum(2)
    # a thread's products in a row, at most H / 256 + 8 of them, then 5 + 8 sums
    close(dw, wl.grad, size * (H / 256 + 24) * 2.0 ** -24)
    assert (dw[r.slots < 0] == 0).all()
    # for one direction at a time, and to other types
    none, dw2 = ops.combine_grad(go, y, r.slots, w, out=False)
    assert none is None and torch.equal(dw, dw2)
    dy2, none = ops.combine_grad(go, None, r.slots, w, out=torch.float32)
    assert none is None
    close(dy2[used], yl.grad[used], yl.grad[used].abs() * 2.0 ** -24)
    for kind in (ops.FP8, ops.MXFP8, ops.NVFP4):
        q, _ = ops.combine_grad(go, y, r.slots, w, out=kind)
        want_q = ops.quantize(dy2, kind)              # of the float32 products: the same bits
        assert torch.equal(q.codes[used], want_q.codes[used]) and torch.equal(q.scales[used], want_q.scales[used])


def test_combine_gradient_against_differences(ops):
    """Central differences of <g, combine> in the weights: it is linear in them, so they are exact but for rounding."""
    r, _ = routes(ops, 9, 4, 12, 3, True)
    g = gen(3)
    y, w = torch.randn(36, 64, device="cuda", generator=g), torch.rand(9, 4, device="cuda", generator=g)
    go = torch.randn(9, 64, device="cuda", generator=g)
    _, dw = ops.combine_grad(go, y, r.slots, w, out=False)
    for t in range(9):
        for j in range(4):
            lo, hi = w.clone(), w.clone()
            lo[t, j] -= 0.5
            hi[t, j] += 0.5
            d = ((ops.combine(y, r.slots, hi).double() - ops.combine(y, r.slots, lo).double()) * go.double()).sum()
            size = (go[t].double().abs() * y.double().abs().amax(0)).sum()
            assert (d - dw[t, j].double()).abs() <= size * 64 * 2.0 ** -24


def test_bad_slots_are_reported_and_skipped(ops):
    x = torch.randn(4, 96, device="cuda")
    slots = torch.tensor([[0, 8], [1, -7], [2, 1 << 30], [3, -1]], dtype=torch.int32, device="cuda")
    good = torch.tensor([[0, -1], [1, -1], [2, -1], [3, -1]], dtype=torch.int32, device="cuda")
    w = torch.rand(4, 2, device="cuda")
    for call, want in ((lambda s, e: ops.dispatch(x, s, out=torch.zeros(8, 96, device="cuda"), error_word=e), None),
                       (lambda s, e: ops.combine(x, s, w, error_word=e), None),
                       (lambda s, e: ops.combine_grad(x, x, s, w, out=torch.zeros(4, 96, device="cuda"), error_word=e)[1], None)):
        word = torch.zeros(1, dtype=torch.int32, device="cuda")
        got, want = call(slots, word), call(good, torch.zeros_like(word))
        assert word.item() != 0 and torch.equal(got, want)
        call(good, word.zero_())
        assert word.item() == 0


def test_rows_strides_and_alignment(ops):
    r, _ = routes(ops, 60, 4, 20, 5, True)
    g = gen(5)
    big = torch.randn(240, 203, device="cuda", generator=g)
    for dtype in DTYPES:
        y, res = big.to(dtype)[:, 1:131], big.to(dtype)[:60, 3:133]
        assert torch.equal(ops.combine(y, r.slots, r.weights, residual=res), ops.combine(y.contiguous(), r.slots, r.weights, residual=res.contiguous()))
        out = torch.zeros(240, 150, dtype=dtype, device="cuda")
        ops.dispatch(res, r.slots, out=out[:, 7:137])
        want = ops.dispatch(res.contiguous(), r.slots, out=torch.zeros(240, 130, dtype=dtype, device="cuda"))
        assert torch.equal(out[:, 7:137], want) and (out[:, :7] == 0).all() and (out[:, 137:] == 0).all()
        dy, dw = ops.combine_grad(res, y, r.slots, r.weights, out=torch.zeros(240, 150, dtype=dtype, device="cuda")[:, 7:137])
        dy2, dw2 = ops.combine_grad(res.contiguous(), y.contiguous(), r.slots, r.weights, out=torch.zeros(240, 130, dtype=dtype, device="cuda"))
        assert torch.equal(dy, dy2) and torch.equal(dw, dw2)


def test_no_tokens(ops):
    x, slots = torch.zeros(0, 64, device="cuda"), torch.zeros(0, 3, dtype=torch.int32, device="cuda")
    assert ops.quantize(x, ops.FP8).codes.shape == (0, 64) and ops.dispatch(x, slots).shape == (0, 64)
    assert ops.combine(x, slots).shape == (0, 64) and ops.combine_grad(x, x, slots)[1].shape == (0, 3)
    assert ops.route_grad(x, slots, slots.float(), slots.float()).shape == (0, 64)
    w, ws = torch.zeros(1, 128, 64, dtype=torch.uint8, device="cuda"), torch.zeros(1, 1, 1, device="cuda")
    assert ops.fp8_matmul(ops.quantize(x, ops.FP8), w, ws).shape == (0, 128)


def test_rows_past_32_bit_offsets(ops):
    S, H = 70000, 32768                               # 2.3e9 elements
    y = torch.zeros(S, H, dtype=torch.float16, device="cuda")
    y[S - 1], y[S - 3] = 1.5, 2.0
    slots = torch.tensor([[S - 1, 0], [S - 3, -1]], dtype=torch.int32, device="cuda")
    out = ops.combine(y, slots)
    assert (out[0] == 1.5).all() and (out[1] == 2).all()
    x = torch.full((2, H), 4.0, dtype=torch.float16, device="cuda")
    ops.dispatch(x, slots, out=y)
    assert (y[S - 1] == 4).all() and (y[S - 3] == 4).all() and (y[S - 2] == 0).all()
    _, dw = ops.combine_grad(x, y, slots, out=False)
    assert dw[0, 0] == 16 * H and dw[1, 0] == 16 * H


# ---- the router's gradient -----------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k,masked", [(1, 1, 1, False), (1, 512, 8, False), (33, 129, 6, True), (300, 40, 8, True), (50, 1024, 32, False), (9, 700, 3, True),
                                          (5000, 256, 8, False), (71, 384, 12, True), (6, 100, 16, False), (3, 390, 5, False)])
def test_route_gradient(ops, T, E, k, masked, renormalize, dtype):
    g = gen(T + E)
    logits = torch.randn(T, E, device="cuda", generator=g)
    if masked:
        logits[torch.rand(T, E, device="cuda", generator=g) < 0.5] = -math.inf
        logits[::3, 2:] = -math.inf
        logits[1::4] = -math.inf
    logits = logits.to(dtype)
    r = ops.route(logits, k, renormalize=renormalize)
    dw = torch.randn(T, k, device="cuda", generator=g)
    out = ops.route_grad(logits, r.ids, r.weights, dw, renormalize=renormalize)
    # by autograd in 64 bits of the weights' definition
    v = torch.where(logits == -math.inf, torch.full((), -1e30, dtype=torch.float64, device="cuda"), logits.double()).requires_grad_()
    on = r.ids >= 0
    p = torch.softmax(v, 1).gather(1, r.ids.clamp(min=0).long())
    p = torch.where(on, p, torch.zeros_like(p))
    if renormalize:
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    (p * torch.where(on, dw, torch.zeros_like(dw)).double()).sum().backward()
    want = torch.nan_to_num(v.grad)
    # terms of up to |w d| and p sum |w d|; the weights are within 2^-20 of theirs, an exponential 2^-18
    size = (r.weights.double() * dw.double().abs() * on).sum(1, keepdim=True)
    near = torch.zeros_like(want).scatter_add_(1, r.ids.clamp(min=0).long(), torch.where(on, r.weights.double() * (dw.double().abs() + size), torch.zeros_like(size)))
    probs = torch.nan_to_num(torch.softmax(logits.double(), 1)) * size
    close(out, want, (near + probs) * 2.0 ** -18)
    assert (out[(r.ids < 0).all(1)] == 0).all()
    same = logits.clone()                             # in place
    ops.route_grad(same, r.ids, r.weights, dw, renormalize=renormalize, out=same)
    assert torch.equal(same, out)
    wide = torch.zeros(T, E + 9, dtype=dtype, device="cuda")
    wide[:, 5:5 + E] = logits                         # rows off 16 bytes
    assert torch.equal(ops.route_grad(wide[:, 5:5 + E], r.ids, r.weights, dw, renormalize=renormalize), out)


def test_route_gradient_against_differences(ops):
    logits = torch.tensor([[1.0, 0.25, -0.5, 2.0, 0.0]], device="cuda")
    dw = torch.tensor([[0.7, -1.1, 0.4]], device="cuda")
    for renormalize in (True, False):
        r = ops.route(logits, 3, renormalize=renormalize)
        d = ops.route_grad(logits, r.ids, r.weights, dw, renormalize=renormalize)
        for e in range(5):
            step = 2.0 ** -6
            up_, down = logits.clone(), logits.clone()
            up_[0, e] += step
            down[0, e] -= step
            a, b = ops.route(up_, 3, renormalize=renormalize), ops.route(down, 3, renormalize=renormalize)
            assert torch.equal(a.ids, r.ids) and torch.equal(b.ids, r.ids)
            slope = ((a.weights - b.weights) * dw).sum() / (2 * step)
            # the third derivative's share of a central difference is step^2 / 6, rounding 2^-22 / step
            assert (slope - d[0, e]).abs() < 2 * step ** 2 + 2.0 ** -14


def test_route_gradient_of_repeated_and_missing_ids(ops):
    logits = torch.randn(2, 9, device="cuda", generator=gen(1))
    ids = torch.tensor([[3, 3, -1], [0, 9, 8]], dtype=torch.int32, device="cuda")
    w, dw = torch.rand(2, 3, device="cuda"), torch.randn(2, 3, device="cuda")
    on = (ids >= 0) & (ids < 9)
    for renormalize in (True, False):
        d = ops.route_grad(logits, ids, w, dw, renormalize=renormalize)
        wd = torch.where(on, w * dw, torch.zeros_like(w)).double()
        dot = wd.sum(1, keepdim=True)
        own = torch.where(on, w.double() * (dw.double() - dot), torch.zeros_like(dot)) if renormalize else wd
        want = torch.zeros(2, 9, dtype=torch.float64, device="cuda") if renormalize else -torch.softmax(logits.double(), 1) * dot
        want.scatter_add_(1, torch.where(on, ids, 0).long(), own)
        close(d, want, 2.0 ** -20 * torch.ones_like(want))


# ---- together ------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("T,masked", [(1, False), (37, True), (300, False)])
def test_a_layer_forwards_and_back(ops, T, masked):
    """Norm, router, 8-bit gate/up and down products and the sum of each token's experts; then the gradients from the
    sum's back to the layer's input and the router's logits.  Each step against 64 bits, from what the steps before
    made."""
    H, I, E, k = 640, 256, 12, 4
    g = gen(T)
    dev = dict(device="cuda", generator=g)
    x = torch.randn(T, H, **dev).to(torch.bfloat16)
    h = torch.randn(T, H, **dev).to(torch.bfloat16)
    w1 = (torch.randn(E, 2 * I, H, **dev) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    w2 = (torch.randn(E, H, I, **dev) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    s1 = (0.5 + torch.rand(E, blocks(2 * I), blocks(H), **dev)) / (100 * H ** 0.5)
    s2 = (0.5 + torch.rand(E, blocks(H), blocks(I), **dev)) / (100 * I ** 0.5)
    q, h = ops.rms_norm(x, torch.ones(H, dtype=torch.bfloat16, device="cuda"), ops.FP8, residual=h)
    logits = torch.randn(T, E, **dev)
    if masked:
        logits[torch.rand(T, E, **dev) < 0.6] = -math.inf
        logits[5::6] = -math.inf
    r = ops.route(logits, k)
    a = ops.fp8_matmul(q, w1, s1, expert_start=r.expert_start, rows=r.rows.clamp(min=0), activation="silu", gated=True, out=ops.FP8)
    y = ops.fp8_matmul(a, w2, s2, expert_start=r.expert_start)
    out = ops.combine(y, r.slots, r.weights, residual=h)

    used = int(r.expert_start[-1])
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), r.expert_start.diff().long())
    rows = r.rows[:used].long()
    wide = lambda s: s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)  # noqa: E731
    v1, v2 = w1.double() * wide(s1), w2.double() * wide(s2)

    def product(x64, w64, transposed=False):          # and its slack
        w = w64[expert]
        w = w if transposed else w.transpose(1, 2)
        depth = w.shape[1]
        return (x64[:, None] @ w)[:, 0], (x64.abs()[:, None] @ w.abs())[:, 0] * (depth / 32 + 4) * 2.0 ** -23

    cut = lambda z: ops.Quantized(z.kind, z.codes[:used], z.scales[:used], z.cols)  # noqa: E731
    p64, slack = product(values(q)[rows], v1)
    gate, upper = p64[:, :I], p64[:, I:]
    eg, eu = slack[:, :I], slack[:, I:]
    act = act64(gate, "silu")
    check_quantized(cut(a), act * upper, (1.1 * eg + act.abs() * 2.0 ** -20) * (upper.abs() + eu) + act.abs() * eu + (act * upper).abs() * 2.0 ** -23)
    y64, slack = product(values(a)[:used], v2)
    close(y[:used], y64, slack)
    want = combine64(torch.where(torch.isfinite(y), y, 0).double(), r.slots, r.weights.double(), h.double())
    size = combine64(torch.where(torch.isfinite(y), y, 0).double().abs(), r.slots, r.weights.double(), h.double().abs())
    close(out, want, size * (k + 2) * 2.0 ** -24)

    # back
    go = torch.randn(T, H, **dev).to(torch.bfloat16)
    dy, dw = ops.combine_grad(go, y, r.slots, r.weights, out=ops.FP8)
    da = ops.fp8_matmul(dy, w2, s2, expert_start=r.expert_start, transposed=True, out=torch.float32)
    p = ops.fp8_matmul(q, w1, s1, expert_start=r.expert_start, rows=r.rows.clamp(min=0), out=torch.float32)
    sg = torch.sigmoid(p[:, :I])
    dp = torch.cat([da * p[:, I:] * sg * (1 + p[:, :I] * (1 - sg)), da * p[:, :I] * sg], 1)
    dp[used:] = 0
    dxs = ops.fp8_matmul(ops.quantize(dp, ops.FP8), w1, s1, expert_start=r.expert_start, transposed=True, out=torch.float32)
    dx = ops.dispatch_grad(dxs, r.slots)
    dl = ops.route_grad(logits, r.ids, r.weights, dw)

    weight = torch.zeros(T * k + 1, device="cuda")
    weight[r.slots.view(-1).long()] = r.weights.view(-1)
    check_quantized(cut(dy), (weight[:used, None] * go[rows].float()).double())
    da64, slack = product(values(dy)[:used], v2, transposed=True)
    close(da[:used], da64, slack)
    # silu(u) v and its derivatives in 64 bits, from the 32-bit sums, against differences
    u, v = p[:used, :I].double(), p[:used, I:].double()
    step = 2.0 ** -12
    slope = (act64(u + step, "silu") - act64(u - step, "silu")) / (2 * step)
    want = torch.cat([da[:used].double() * v * slope, da[:used].double() * act64(u, "silu")], 1)
    assert ((dp[:used].double() - want).abs() <= want.abs() * 2.0 ** -18 + (da[:used].double().abs() * v.abs()).repeat(1, 2) * 2.0 ** -18).all()
    dx64, slack = product(values(ops.quantize(dp, ops.FP8))[:used], v1, transposed=True)
    close(dxs[:used], dx64, slack)
    sums, size = torch.zeros(T, H, dtype=torch.float64, device="cuda"), torch.zeros(T, H, dtype=torch.float64, device="cuda")
    sums.index_add_(0, rows, dxs[:used].double())
    size.index_add_(0, rows, dxs[:used].double().abs())
    close(dx, sums, size * k * 2.0 ** -24)
    w64, dw64 = r.weights.double(), dw.double()
    own = w64 * (dw64 - (w64 * dw64).sum(1, keepdim=True))
    want = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_add_(1, r.ids.clamp(min=0).long(), torch.where(r.ids >= 0, own, 0))
    bound = (w64 * (dw64.abs() + (w64 * dw64.abs()).sum(1, keepdim=True))).sum(1, keepdim=True)
    close(dl, want, bound * 2.0 ** -20)


def test_inputs_may_be_let_go_of_and_capture_beside_eager_calls(ops):
    """Calls on another stream keep their inputs; a captured run of the operators replays beside eager ones."""
    r, _ = routes(ops, 64, 4, 16, 1, False)
    g = gen(2)
    p = Problem(ops, [256], 256, 512, seed=3)
    side = torch.cuda.Stream()
    want = ops.combine(p.run(out=torch.float32), r.slots, r.weights)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    y = p.run(out=torch.float32, stream=side)
    out = ops.combine(y, r.slots, r.weights, stream=side)
    del y
    torch.randn(1 << 22, device="cuda", generator=g)   # memory that is taken again meanwhile
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    ops.errors()                                       # the device's word, before a capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = p.run(out=torch.float32)
        out = ops.combine(y, r.slots, r.weights)
        dy, dw = ops.combine_grad(out, y, r.slots, r.weights, out=ops.FP8)
        back = ops.fp8_matmul(dy, p.w, p.ws, transposed=True)
    eager = p.run(out=torch.float32)
    graph.replay()
    eager2 = p.run(out=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(eager, eager2) and torch.equal(out, want)
    dy2, dw2 = ops.combine_grad(want, eager, r.slots, r.weights, out=ops.FP8)
    assert torch.equal(dw, dw2) and torch.equal(dy.codes, dy2.codes) and torch.equal(back, ops.fp8_matmul(dy2, p.w, p.ws, transposed=True))
