"""The expert-layer operators against their definitions in 64 bits.

Tolerances come from the arithmetic, before any run:
  sums       a product's sum is held in 32 bits over K/32 matrix steps, each
             off by at most 2^-23 of what it holds, itself at most S = sum |x w|;
             with the operands exact the error is at most (K/32 + 4) 2^-23 S.
  epilogue   a handful of 32-bit operations, 2^-20 of the magnitudes involved;
             activations have slopes below 1.13.
  types      half a unit in the last place of bfloat16 (2^-9) or float16 (2^-12).
  codes      a code is the nearest one to the value, so it is off by half the
             distance to its neighbour, more only by the value's own error.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF_ULP = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 0.0}    # of the value, doubled for values at a binade's low end


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_nvfp4_scale_gb300 import build
    build.ensure_built()
    from lossless_nvfp4_scale_gb300 import ops as mod
    return mod


def up(n, m):
    return -(-n // m) * m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def unpack(codes):
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    return torch.stack([t[(codes & 15).long()], t[(codes >> 4).long()]], -1).flatten(-2)


def scale_values(b, kind, ops):
    if kind == ops.NVFP4:
        return b.view(torch.float8_e4m3fn).double()
    v = torch.exp2(b.double() - 127)
    return torch.where(b == 255, torch.full_like(v, math.nan), v)


def code_values(q, ops):
    v = unpack(q.codes) if q.kind == ops.NVFP4 else q.codes.view(torch.float8_e4m3fn).double()
    return v[:, :up(q.cols, 32)]


def values(q, ops):
    """A quantised tensor as the values it stands for, [rows, cols padded to 32]."""
    block = 16 if q.kind == ops.NVFP4 else 32
    cols = up(q.cols, 32)
    s = scale_values(q.scales[:, :cols // block], q.kind, ops)
    v = (code_values(q, ops).view(q.rows, cols // block, block) * s[..., None]).view(q.rows, cols)
    return v * q.tensor_scale.double() if q.tensor_scale is not None else v


def check_quantized(q, y, err, ops):
    """q holds the nearest codes of y [rows, cols], known to within err (same shape)."""
    block = 16 if q.kind == ops.NVFP4 else 32
    cols = up(q.cols, 32)
    g = q.tensor_scale.double() if q.tensor_scale is not None else 1.0
    pad = lambda v: torch.nn.functional.pad(v, (0, cols - q.cols)).view(q.rows, -1, block)  # noqa: E731
    y, err = pad(y), pad(err)
    s = scale_values(q.scales[:, :cols // block], q.kind, ops)
    lo, hi = (y.abs() - err).amax(2).clamp(min=0), (y.abs() + err).amax(2)
    if q.kind == ops.MXFP8:
        assert (448 * s >= lo * (1 - 1e-12)).all()
        assert ((224 * s < hi * (1 + 1e-12)) | (s == 2.0 ** -127)).all()     # no smaller power of two would do
    else:
        near = lambda v: (v / (6 * g)).clamp(max=448).float().to(torch.float8_e4m3fn).double()  # noqa: E731
        assert ((s >= near(lo * (1 - 2.0 ** -22))) & (s <= near(hi * (1 + 2.0 ** -22)))).all()
    whole = (s * g)[..., None]
    c = code_values(q, ops).view(q.rows, -1, block)
    v = torch.where(whole > 0, y / whole, torch.zeros_like(y))
    slack = torch.where(whole > 0, err / whole, torch.zeros_like(y)) + 2.0 ** -20 * v.abs()
    if q.kind == ops.MXFP8:
        exp = torch.frexp(c.abs().clamp(min=2.0 ** -6)).exponent - 1
        half = torch.ldexp(torch.ones_like(c), exp - 4)
    else:
        a = c.abs()
        half = torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, 1.0)).to(v.dtype)
        v = v.clamp(-6, 6)
    assert ((c - v).abs() <= half + slack).all()
    blocks = cols // block
    assert (q.scales[:, blocks:up(blocks, 16)] == 0).all()                   # the scale row's padding
    assert (code_values(q, ops)[:, q.cols:] == 0).all()


# ---- rms_norm --------------------------------------------------------------------------------------------------------

def norm_reference(x, w, residual, eps):
    h = x.double() + (residual.double() if residual is not None else 0)
    return h, h / ((h * h).mean(1, keepdim=True) + eps).sqrt() * w.double()


def check_norm(q, total, x, w, residual, eps, ops):
    h, y = norm_reference(x, w, residual, eps)
    check_quantized(q, y, y.abs() * 2.0 ** -18, ops)
    if residual is not None:
        assert ((total.double() - h).abs() <= HALF_ULP[x.dtype] * h.abs() + 2.0 ** -24 * (x.double().abs() + residual.double().abs()) + 2.0 ** -25).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 32), (7, 33), (9, 256), (5, 257), (2, 1001), (4, 1600),
                                       (3, 5120), (2, 16384), (2, 16385), (1, 40000)])
def test_norm(ops, rows, cols, kind, dtype):
    g = gen(rows * 100003 + cols)
    x = torch.randn(rows, cols, device="cuda", generator=g).to(dtype)
    r = torch.randn(rows, cols, device="cuda", generator=g).to(dtype) if cols % 2 else None
    w = (1 + 0.3 * torch.randn(cols, device="cuda", generator=g)).to(dtype)
    ts = torch.tensor([0.02], device="cuda") if kind == ops.NVFP4 else None
    q, total = ops.rms_norm(x, w, kind, residual=r, eps=1e-5, tensor_scale=ts)
    check_norm(q, total, x, w, r, 1e-5, ops)


@pytest.mark.parametrize("kind", [0, 1])
def test_norm_strides_alignment_and_in_place_sum(ops, kind):
    g = gen(5)
    for cols, width, off in ((100, 131, 1), (320, 336, 8), (320, 321, 0)):
        big = torch.randn(3, 6, width, device="cuda", generator=g).to(BF16)
        x, r = big[0, :, off:off + cols], big[1, :, off:off + cols]
        w = torch.randn(cols + 1, device="cuda", generator=g).to(BF16)[1:]
        x0, r0 = x.clone(), r.clone()
        outside = big.clone()
        q, total = ops.rms_norm(x, w, kind, residual=r, sum_out=r)           # the residual stream updated in place
        assert total is r
        check_norm(q, r, x0, w, r0, 1e-6, ops)
        outside[1, :, off:off + cols] = r
        assert torch.equal(outside.view(torch.int16), big.view(torch.int16))  # nothing else was written
        x1 = x.clone()
        q2, _ = ops.rms_norm(x1, w, kind, residual=r0.contiguous(), sum_out=x1)
        check_norm(q2, x1, x0, w, r0, 1e-6, ops)
        assert torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales)


def test_norm_wide_rows_sum_in_place(ops):
    x, r = torch.randn(2, 20000, device="cuda", generator=gen(1)), torch.randn(2, 20000, device="cuda", generator=gen(2))
    w = torch.ones(20000, device="cuda")
    r0 = r.clone()
    q, total = ops.rms_norm(x, w, ops.MXFP8, residual=r, sum_out=r)
    check_norm(q, total, x, w, r0, 1e-6, ops)


@pytest.mark.parametrize("kind", [0, 1])
def test_norm_zero_huge_and_non_finite_rows(ops, kind):
    x = torch.zeros(5, 64, device="cuda")
    x[1, 3] = 1e-30
    x[2, 5] = 3e37
    x[3, 40] = math.inf
    x[4, 7] = math.nan
    w = torch.ones(64, device="cuda")
    q, _ = ops.rms_norm(x, w, kind, eps=1e-6)
    block = 16 if kind == ops.NVFP4 else 32
    s = scale_values(q.scales[:, :64 // block], kind, ops)
    assert (code_values(q, ops)[0] == 0).all() and torch.isfinite(s[:2]).all()
    assert (values(q, ops)[:2] == 0).all() or kind == ops.MXFP8
    assert torch.isnan(s[3, 40 // block])                     # inf * (1 / inf) is NaN in its own block
    assert torch.isnan(s[4]).all()                            # a NaN reaches the whole row through its mean


def test_norm_no_rows(ops):
    q, total = ops.rms_norm(torch.zeros(0, 64, device="cuda"), torch.ones(64, device="cuda"), ops.NVFP4,
                            residual=torch.zeros(0, 64, device="cuda"))
    assert q.rows == 0 and total.shape == (0, 64)


# ---- route -----------------------------------------------------------------------------------------------------------

def check_route(r, logits, k, renormalize):
    T, E = logits.shape
    v = logits.double()
    ids = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :k]      # ties to the lower expert
    chosen = v.gather(1, ids)
    on = ~(chosen == -math.inf)
    ids = torch.where(on, ids, torch.full_like(ids, -1))
    assert torch.equal(r.ids.long(), ids)
    p = torch.softmax(v, 1).gather(1, ids.clamp(min=0))
    p = torch.where(on, p, torch.zeros_like(p))
    if renormalize:
        z = torch.exp(chosen - chosen[:, :1])
        z = torch.where(on, z, torch.zeros_like(z))
        p = torch.where(on, z / z.sum(1, keepdim=True), torch.zeros_like(z))
    same_nan = torch.isnan(p) == torch.isnan(r.weights.double())
    assert same_nan.all()
    ok = ~torch.isnan(p)
    # exp of a difference of up to 2^7 held in 32 bits, a sum of E terms, one division
    assert ((r.weights.double() - p).abs()[ok] <= (2.0 ** -17 + E * 2.0 ** -24) * p[ok] + 1e-38).all()
    flat = torch.where(ids < 0, torch.full_like(ids, E), ids).reshape(-1)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    start = torch.cat([torch.zeros(1, dtype=torch.long, device=v.device), counts.cumsum(0)])
    assert torch.equal(r.expert_start.long(), start)
    slot_of = torch.argsort(flat, stable=True)
    used = int(start[-1])
    assert torch.equal(r.rows.long()[:used], (slot_of // k)[:used])
    assert (r.rows[used:] == -1).all()
    slots = torch.full_like(flat, -1)
    slots[slot_of[:used]] = torch.arange(used, device=v.device)
    assert torch.equal(r.slots.long().reshape(-1), slots)


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T,E,k,dtype", [(1, 1, 1, F32), (1, 512, 8, F32), (2, 33, 32, BF16), (63, 129, 6, F16),
                                         (64, 1024, 8, F32), (65, 1024, 3, BF16), (129, 7, 7, F32), (1000, 256, 2, F32),
                                         (4097, 60, 4, BF16)])
def test_route(ops, T, E, k, dtype, renormalize):
    logits = (2 * torch.randn(T, E, device="cuda", generator=gen(T + E))).to(dtype)
    check_route(ops.route(logits, k, renormalize=renormalize), logits, k, renormalize)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,E", [(40, 40), (200, 40), (70, 501), (600, 501), (1000, 130)])
def test_route_ties_masks_and_empty_rows(ops, T, E, dtype):
    k = 6
    v = torch.randint(-2, 3, (T, E), device="cuda", generator=gen(T)).to(dtype)   # many ties
    v[::3, 5:] = -math.inf                                                        # fewer experts than k
    v[::7] = -math.inf                                                            # none left
    v[1, 3], v[1, 9] = 0.0, -0.0                                                  # equal zeros
    v[2, 4] = torch.finfo(dtype).min                                               # the lowest number is no mask
    v[2, 5:] = -math.inf
    check_route(ops.route(v, k, renormalize=True), v, k, True)
    r = ops.route(v, k, renormalize=False)
    assert torch.isfinite(r.weights).all()
    assert (r.weights[::7] == 0).all() and (r.ids[::7] == -1).all() and (r.slots[::7] == -1).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_route_non_finite(ops, dtype):
    v = torch.randn(70, 30, device="cuda", generator=gen(3)).to(dtype)
    v[5, 3], v[6, 3] = -math.nan, math.nan
    v[5:7].view(torch.int16 if dtype is not F32 else torch.int32)[0, 3] |= -0x8000 if dtype is not F32 else -0x80000000
    v[0, 7] = math.nan
    v[1, 7] = math.inf
    v[66, 2] = math.nan
    v[66, 9] = math.inf
    r = ops.route(v, 4)
    assert r.ids[0, 0] == 7 and r.ids[1, 0] == 7 and r.ids[66, :2].tolist() == [2, 9]
    assert torch.isnan(r.weights[0]).all() and torch.isnan(r.weights[66]).all()
    clean = torch.ones(70, dtype=torch.bool, device="cuda")
    assert r.ids[5, 0] == 3 and r.ids[6, 0] == 3                  # a NaN of either sign
    clean[[0, 1, 5, 6, 66]] = False
    assert torch.isfinite(r.weights[clean]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("width,off", [(150, 11), (151, 10), (152, 16)])
def test_route_strided_logits_no_tokens_and_repeats(ops, width, off, dtype):
    big = torch.randn(600, width, device="cuda", generator=gen(9)).to(dtype)
    v = big[:, off:off + 101]
    a, b = ops.route(v, 5), ops.route(v, 5)
    check_route(a, v, 5, True)
    for f in ("ids", "weights", "expert_start", "rows", "slots"):
        assert torch.equal(getattr(a, f), getattr(b, f))
    r = ops.route(big[:0], 5)
    assert r.ids.shape == (0, 5) and (r.expert_start == 0).all()


# ---- expert_matmul ---------------------------------------------------------------------------------------------------

def blocked(scales):
    E, N, C = scales.shape
    p = torch.zeros(E, up(N, 128), up(C, 4), dtype=torch.uint8, device=scales.device)
    p[:, :N, :C] = scales
    return p.view(E, -1, 4, 32, p.shape[2] // 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(-1)


class Problem:
    def __init__(self, ops, kind, counts, N, K, seed=0, gather=0, tail=0, out_cols=None):
        g = gen(seed * 7919 + N + K)
        self.ops, self.kind, self.N, self.K, self.E = ops, kind, N, K, len(counts)
        self.counts, self.used = counts, sum(counts)
        self.S = self.used + tail                              # slots past the last expert's end
        self.T = gather or self.S
        dev = dict(device="cuda", generator=g)
        block = 16 if kind == ops.NVFP4 else 32
        lo, hi = (0x20, 0x40) if kind == ops.NVFP4 else (122, 130)
        codes = torch.randint(0, 256, (self.T, K // 2 if kind == ops.NVFP4 else K), dtype=torch.uint8, **dev)
        if kind == ops.MXFP8:
            codes = (codes & 0x80) | ((codes & 0x7F) % 0x50)   # up to 2^3, subnormals among them
        scales = torch.zeros(self.T, up(K // block, 16), dtype=torch.uint8, device="cuda")
        scales[:, :K // block] = torch.randint(lo, hi, (self.T, K // block), dtype=torch.uint8, **dev)
        self.x = ops.Quantized(kind, codes, scales, K)
        self.w = torch.randint(0, 256, (self.E, N, K // 2), dtype=torch.uint8, **dev)
        ws = torch.randint(lo, hi, (self.E, N, K // block), dtype=torch.uint8, **dev)
        self.ws = blocked(ws)
        self.start = torch.tensor([sum(counts[:i]) for i in range(self.E + 1)], dtype=torch.int32, device="cuda")
        self.rows = torch.randint(0, self.T, (self.S,), dtype=torch.int32, **dev) if gather else None
        self.alpha = 0.01 + 0.02 * torch.rand(self.E, **dev)
        self.dev = dev
        x = values(self.x, ops)
        x = x[self.rows.long()] if gather else x
        w = (unpack(self.w).view(self.E, N, -1, block) * scale_values(ws, kind, ops)[..., None]).view(self.E, N, K)
        self.p = torch.zeros(self.S, N, dtype=torch.float64, device="cuda")
        self.mag = torch.zeros_like(self.p)
        at = 0
        self.e = torch.zeros(self.S, dtype=torch.long, device="cuda")
        for e, c in enumerate(counts):
            self.p[at:at + c] = x[at:at + c] @ w[e].T
            self.mag[at:at + c] = x[at:at + c].abs() @ w[e].T.abs()
            self.e[at:at + c] = e
            at += c

    def expect(self, act=None, gated=False, alpha=None, bias=None, row_scale=None, residual=None):
        """The result in 64 bits and how far the kernel's may be from it."""
        a = (alpha.double()[self.e] if alpha is not None else torch.ones(self.S, dtype=torch.float64, device="cuda"))[:, None]
        p = self.p * a
        err = (self.K / 32 + 4) * 2.0 ** -23 * self.mag * a
        if bias is not None:
            b = bias.double()[self.e]
            p, err = p + b, err + 2.0 ** -22 * b.abs()
        f = {None: lambda v: v, "relu": lambda v: v.clamp(min=0), "silu": lambda v: v * torch.sigmoid(v),
             "gelu": lambda v: v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))}[act]
        if gated:
            n = self.N // 2
            left, right = f(p[:, :n]), p[:, n:]
            el = 1.13 * err[:, :n] + 2.0 ** -19 * p[:, :n].abs()
            y = left * right
            err = el * right.abs() + left.abs() * err[:, n:] + el * err[:, n:]
        else:
            y, err = f(p), 1.13 * err + (2.0 ** -19 * p.abs() if act else 0)
        if row_scale is not None:
            y, err = y * row_scale.double()[:, None], err * row_scale.double().abs()[:, None]
        err = err + 2.0 ** -22 * y.abs()
        if residual is not None:
            y, err = y + residual.double(), err + 2.0 ** -23 * residual.double().abs()
        return y, err

    def run(self, **kw):
        kw.setdefault("expert_start", self.start)
        return self.ops.expert_matmul(self.x, self.w, self.ws, rows=self.rows, **kw)

    def check(self, out, **kw):
        y, err = self.expect(**kw)
        u = self.used
        if isinstance(out, torch.Tensor):
            top = torch.finfo(out.dtype).max
            over = (y.abs() - err > top * (1 + HALF_ULP[out.dtype]))[:u]         # rounds to an infinity of its sign
            assert (out[:u][over].double() == torch.sign(y[:u][over]) * math.inf).all()
            y = torch.where(y.abs() + err > top, out.double(), y)
            bound = err + HALF_ULP[out.dtype] * y.abs() + (2.0 ** -24 if out.dtype == F16 else 0)
            assert ((out.double() - y).abs() <= bound)[:u][~over].all()
        else:
            cut = self.ops.Quantized(out.kind, out.codes[:u], out.scales[:u], out.cols, out.tensor_scale)
            check_quantized(cut, y[:u], err[:u], self.ops)


SHAPES = [  # counts, N, K in 32s (NVFP4) or 128s (MXFP8), gathered rows
    ([1], 1, 1, 0), ([1], 128, 4, 0), ([0], 64, 2, 0), ([3], 129, 3, 0), ([16], 64, 8, 5), ([17], 300, 25, 0),
    ([0, 0, 5, 0], 72, 9, 3), ([1, 1, 1, 1, 1, 1, 1], 200, 5, 2), ([129, 0, 300, 1], 136, 12, 64), ([97, 33], 512, 10, 0),
    ([500], 256, 17, 0), ([449, 225], 100, 3, 0)]


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("counts,N,k,gather", SHAPES)
def test_matmul(ops, counts, N, k, gather, kind):
    q = Problem(ops, kind, counts, N, k * (32 if kind == ops.NVFP4 else 128), gather=gather)
    out = q.run(out=F32)
    assert out.shape == (q.S, N)
    q.check(out)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("out", [BF16, F16, F32, "nvfp4", "mxfp8"])
@pytest.mark.parametrize("act,gated", [(None, False), ("relu", False), ("gelu", False), ("silu", True), (None, True),
                                       ("relu", True)])
def test_matmul_epilogue(ops, act, gated, out, kind):
    q = Problem(ops, kind, [3, 0, 40, 131], 512 if gated else 200, 384, seed=3, gather=50)
    bias = torch.randn(q.E, q.N, **q.dev).to(out if isinstance(out, torch.dtype) else BF16)
    F = q.N // 2 if gated else q.N
    row_scale = torch.rand(q.S, **q.dev)
    residual = torch.randn(q.S, F, **q.dev).to(F16 if out is BF16 else F32 if out is F32 else BF16)
    kw = dict(alpha=q.alpha, bias=bias, row_scale=row_scale, residual=residual)
    o = out if isinstance(out, torch.dtype) else ops.NVFP4 if out == "nvfp4" else ops.MXFP8
    ts = torch.tensor([0.004], device="cuda") if out == "nvfp4" else None
    q.check(q.run(out=o, out_tensor_scale=ts, activation=act, gated=gated, **kw), act=act, gated=gated, **kw)
    q.check(q.run(out=o, out_tensor_scale=ts, activation=act, gated=gated), act=act, gated=gated)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("counts,N,K,gather", [([1], 256, 5120, 0), ([1], 2048, 5120, 0), ([16], 256, 1664, 3), ([17], 512, 2048, 0),
                                               ([2, 0, 9], 256, 2176, 4), ([1] * 8, 256, 1664, 1), ([100], 256, 4096, 0)])
def test_matmul_of_few_slots_with_k_shared_by_clusters(ops, counts, N, K, gather, kind):
    q = Problem(ops, kind, counts, N, K, seed=15, gather=gather)
    bias, residual = torch.randn(q.E, N, **q.dev), torch.randn(q.S, N, **q.dev)
    q.check(q.run(out=F32, alpha=q.alpha, bias=bias), alpha=q.alpha, bias=bias)
    q.check(q.run(out=BF16, alpha=q.alpha, residual=residual), alpha=q.alpha, residual=residual)
    q.check(q.run(out=F32, alpha=q.alpha, activation="silu", gated=True), act="silu", gated=True, alpha=q.alpha)
    first = q.run(out=ops.MXFP8)
    q.check(first)
    for _ in range(3):
        again = q.run(out=ops.MXFP8)
        assert torch.equal(first.codes, again.codes) and torch.equal(first.scales, again.scales)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("N", [33, 64, 250])
def test_matmul_ragged_quantized_outputs(ops, N, kind):
    q = Problem(ops, kind, [5, 70], N, 256, seed=4)
    for o in (ops.NVFP4, ops.MXFP8):
        out = ops.empty_quantized(o, q.S, N)
        out.codes.fill_(0xA5)
        out.scales.fill_(0xA5)
        q.check(q.run(out=out, alpha=q.alpha), alpha=q.alpha)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_matmul_strided_and_unaligned_output_and_residual(ops, dtype):
    q = Problem(ops, ops.NVFP4, [20, 37], 101, 320, seed=5)
    for width, off in ((101, 0), (118, 1), (128, 8)):
        big = torch.full((q.S + 2, width), 7.0, device="cuda", dtype=dtype)
        res = torch.randn(q.S, width, **q.dev).to(dtype)[:, off:off + 101]
        out = big[1:-1, off:off + 101]
        q.check(q.run(out=out, alpha=q.alpha, residual=res), alpha=q.alpha, residual=res)
        mask = torch.ones_like(big, dtype=torch.bool)
        mask[1:-1, off:off + 101] = False
        assert (big[mask] == 7.0).all()
    # the residual updated in place
    res = torch.randn(q.S, 101, **q.dev).to(dtype)
    before = res.clone()
    q.check(q.run(out=res, residual=res, alpha=q.alpha), alpha=q.alpha, residual=before)


def test_matmul_strided_x_rows(ops):
    q = Problem(ops, ops.NVFP4, [30], 64, 96, seed=6)
    codes = torch.zeros(30, 80, dtype=torch.uint8, device="cuda")
    scales = torch.full((30, 48), 0x7F, dtype=torch.uint8, device="cuda")        # NaN outside the rows
    codes[:, :48], scales[:, :16] = q.x.codes, q.x.scales
    q.x = ops.Quantized(ops.NVFP4, codes[:, :48], scales[:, :16], 96)
    q.check(q.run(out=F32))


@pytest.mark.parametrize("gather", [0, 9])
def test_matmul_int64_start_and_unowned_slots(ops, gather):
    q = Problem(ops, ops.MXFP8, [4, 0, 21], 72, 256, seed=7, gather=gather, tail=13)
    out = torch.full((q.S, 72), 5.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.check(q.run(out=out, expert_start=q.start.long(), error_word=err))
    assert (out[q.used:] == 5.0).all() and int(err) == 0


def test_matmul_reports_bad_indices_and_starts(ops):
    from lossless_nvfp4_scale_gb300 import csf
    q = Problem(ops, ops.NVFP4, [6, 7], 64, 64, seed=8, gather=5)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q.rows[3], q.rows[8] = 5, -1                                   # x has rows 0 .. 4
    q.run(error_word=err)
    assert int(err) == csf.DEV_ERR_CORRUPT
    for bad in ([0, 6, 14], [0, 7, 5], [-1, 6, 13]):               # past the slots, decreasing, negative
        q = Problem(ops, ops.NVFP4, [6, 7], 64, 64, seed=8)
        err.zero_()
        out = q.run(expert_start=torch.tensor(bad, dtype=torch.int32, device="cuda"), error_word=err)
        assert int(err) & csf.DEV_ERR_CORRUPT, bad
        assert out.shape == (13, 64)


@pytest.mark.parametrize("bad", [[0, 6, 14], [0, 7, 5], [-1, 6, 13], [0, 14, 13], [9, 3, 13]])
@pytest.mark.parametrize("K", [64, 5120])
def test_matmul_writes_nothing_for_a_bad_start(ops, bad, K):
    from lossless_nvfp4_scale_gb300 import csf
    for int64 in (False, True):
        q = Problem(ops, ops.NVFP4, [6, 7], 64, K, seed=8)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((13, 64), 5.0, device="cuda")
        start = torch.tensor(bad, dtype=torch.int64 if int64 else torch.int32, device="cuda")
        q.run(out=out, expert_start=start, error_word=err)
        assert int(err) == csf.DEV_ERR_CORRUPT and (out == 5.0).all()


def test_errors_of_calls_without_an_error_word(ops):
    from lossless_nvfp4_scale_gb300 import csf
    q = Problem(ops, ops.NVFP4, [6, 7], 64, 64, seed=8, gather=5)
    ops.errors()
    q.run()
    assert ops.errors() == 0
    q.rows[2] = 99
    q.run()
    assert ops.errors() == csf.DEV_ERR_CORRUPT and ops.errors() == 0


def test_matmul_no_slots(ops):
    q = Problem(ops, ops.NVFP4, [0, 0], 64, 64)
    assert q.run().shape == (0, 64)
    assert q.run(out=ops.MXFP8).rows == 0


def test_matmul_one_expert_takes_all_and_many_experts(ops):
    q = Problem(ops, ops.NVFP4, [0] * 300 + [700] + [0] * 211, 64, 64, seed=9, gather=100)
    q.check(q.run(out=F32))
    q = Problem(ops, ops.MXFP8, [i % 3 for i in range(700)], 40, 128, seed=10, gather=100)
    q.check(q.run(out=F32))


def test_matmul_without_expert_start(ops):
    q = Problem(ops, ops.MXFP8, [260], 192, 384, seed=11)
    a, b = q.run(out=F32, expert_start=None), q.run(out=F32)
    assert torch.equal(a, b)
    q.check(a)


def test_matmul_non_finite_blocks_stay_in_their_slots(ops):
    """A NaN scale of one x row makes that row's output NaN and no other's."""
    q = Problem(ops, ops.MXFP8, [40], 64, 256, seed=12)
    clean = q.run(out=F32)
    q.x.scales[7, 3] = 255
    out = q.run(out=F32)
    assert torch.isnan(out[7]).all()
    keep = [i for i in range(40) if i != 7]
    assert torch.equal(out[keep], clean[keep])


def test_matmul_repeats_are_equal_bit_for_bit(ops):
    q = Problem(ops, ops.NVFP4, [50, 3, 170], 256, 1600, seed=13, gather=99)
    first = q.run(gated=True, activation="silu")
    for _ in range(5):
        assert torch.equal(first, q.run(gated=True, activation="silu"))


def test_other_stream_and_graph(ops):
    """Calls on a side stream, and a captured layer replayed on new inputs."""
    side = torch.cuda.Stream()
    q = Problem(ops, ops.NVFP4, [30, 50], 256, 320, seed=14)
    side.wait_stream(torch.cuda.current_stream())
    out = q.run(out=F32, stream=side)
    x = torch.randn(80, 320, **q.dev)
    w = torch.ones(320, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    qx, _ = ops.rms_norm(x, w, ops.NVFP4, stream=side)
    r = ops.route(x[:, :64], 4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    q.check(out)
    check_norm(qx, None, x, w, None, 1e-6, ops)
    check_route(r, x[:, :64], 4, True)

    def layer():
        a, _ = ops.rms_norm(x, w, ops.NVFP4)
        return ops.expert_matmul(a, q.w, q.ws, expert_start=q.start, out=F32)

    with torch.cuda.stream(side):
        layer()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = layer()
    x.copy_(torch.randn(80, 320, **q.dev))
    want = layer()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, want)


def test_binding_refusals(ops):
    q = Problem(ops, ops.NVFP4, [8], 64, 64)
    with pytest.raises(ops.CsfError, match="activation"):
        q.run(activation="tanh")
    with pytest.raises(ops.CsfError, match="E.1 entries"):
        q.run(expert_start=q.start[:1])
    with pytest.raises(ops.CsfError, match="residual"):
        q.run(residual=torch.zeros(8, 63, device="cuda"))
    with pytest.raises(ops.CsfError, match="alpha"):
        q.run(alpha=torch.ones(2, device="cuda"))
    with pytest.raises(ops.CsfError, match="w_scales"):
        ops.expert_matmul(q.x, q.w, q.ws[:-1])
    with pytest.raises(ops.CsfError, match="w must be"):
        ops.expert_matmul(q.x, q.w[:, :, :16], q.ws)
    with pytest.raises(ops.CsfError, match="unsupported"):
        q.run(gated=True)
    with pytest.raises(ops.CsfError, match="out"):
        q.run(out=torch.zeros(8, 65, device="cuda"))
    with pytest.raises(ops.CsfError, match="tensor scale"):
        ops.rms_norm(torch.zeros(1, 32, device="cuda"), torch.ones(32, device="cuda"), ops.MXFP8,
                     tensor_scale=torch.ones(1, device="cuda"))


# ---- offsets past 32 bits --------------------------------------------------------------------------------------------

def test_norm_past_32_bits(ops):
    rows, cols = 560_000, 4096                                    # 2.29e9 elements
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    x.normal_(generator=gen(1))
    w = torch.ones(cols, device="cuda", dtype=BF16)
    q, _ = ops.rms_norm(x, w, ops.MXFP8)
    at = torch.tensor([0, 1, 262_143, 524_287, 524_288, rows - 1], device="cuda")
    part = ops.Quantized(ops.MXFP8, q.codes[at], q.scales[at], cols)
    check_norm(part, None, x[at], w, None, 1e-6, ops)


def test_route_past_32_bits(ops):
    T, E, k = 2_200_000, 1000, 2                                  # 2.2e9 logits
    v = torch.empty(T, E, dtype=BF16, device="cuda")
    v.normal_(generator=gen(2))
    r = ops.route(v, k)
    at = torch.tensor([0, 63, 64, 2_147_483, 2_147_484, T - 1], device="cuda")
    part = torch.sort(v[at].double(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.ids[at].long(), part)
    # every choice has a slot of its expert, and slots are in token order
    assert int(r.expert_start[-1]) == T * k
    slots = r.slots.long().view(-1)
    assert torch.equal(r.rows[slots].long(), torch.arange(T, device="cuda").repeat_interleave(k))
    assert torch.equal(torch.searchsorted(r.expert_start[1:].long(), slots, right=True), r.ids.long().view(-1))
    step = r.rows[1:] > r.rows[:-1]
    first = torch.zeros(T * k, dtype=torch.bool, device="cuda")
    first[r.expert_start[:-1].long().clamp(max=T * k - 1)] = True
    assert (step | first[1:]).all()


def test_matmul_past_32_bits(ops):
    S, N, K = 70_000, 40_000, 64                                  # 2.8e9 outputs
    q = Problem(ops, ops.NVFP4, [4], N, K, seed=20)
    g = gen(21)
    codes = torch.randint(0, 256, (S, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.zeros(S, 16, dtype=torch.uint8, device="cuda")
    scales[:, :4] = torch.randint(0x20, 0x40, (S, 4), dtype=torch.uint8, device="cuda", generator=g)
    at = torch.tensor([0, 53_687, 53_688, S - 1], device="cuda")   # 53687.09 rows reach 2^31 outputs
    codes[at], scales[at] = q.x.codes, q.x.scales
    residual = torch.empty(S, N, dtype=BF16, device="cuda")
    residual.normal_(generator=g)
    out = ops.expert_matmul(ops.Quantized(ops.NVFP4, codes, scales, K), q.w, q.ws, residual=residual)
    q.check(out[at], residual=residual[at])


@pytest.mark.parametrize("act,plus,minus", [(None, math.inf, -math.inf), ("relu", math.inf, 0.0), ("silu", math.inf, math.nan),
                                            ("gelu", math.inf, math.nan)])
def test_matmul_infinite_sums(ops, act, plus, minus):
    """An infinite bias makes its own column what the formula makes of it, large ones saturate the sigmoid."""
    q = Problem(ops, ops.NVFP4, [5], 64, 64, seed=16)
    bias = torch.zeros(1, 64, device="cuda")
    bias[0, 3], bias[0, 4], bias[0, 5], bias[0, 6] = math.inf, -math.inf, 1e30, -1e30
    out = q.run(out=F32, bias=bias, activation=act)
    assert (out[:, 3] == plus).all()
    assert (torch.isnan(out[:, 4]) if math.isnan(minus) else out[:, 4] == minus).all()
    keep = [i for i in range(64) if i not in (3, 4, 5, 6)]
    assert torch.isfinite(out[:, keep]).all()
    assert ((out[:, 5] - 1e30).abs() <= 1e24).all()
    assert (out[:, 6] == -1e30).all() if act is None else (out[:, 6].abs() <= 1e-5).all()


@pytest.mark.parametrize("kind,K", [(0, 4096), (1, 2048)])
def test_matmul_one_slot_of_8192_experts(ops, kind, K):
    """The most experts, one of them with a slot: their prefixes leave little shared memory for a cluster's sums."""
    E, N, e = 8192, 256, 8190
    q = Problem(ops, kind, [1], N, K, seed=17)
    w = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(E, q.ws.numel(), dtype=torch.uint8, device="cuda")
    w[e], ws[e] = q.w[0], q.ws
    start = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    start[e + 1:] = 1
    for kw in (dict(out=F32), dict(out=F32, gated=True, activation="silu")):
        out = ops.expert_matmul(q.x, w, ws.view(-1), expert_start=start, **kw)
        q.check(out, act=kw.get("activation"), gated=kw.get("gated", False))
    assert ops.errors() == 0
    many = torch.zeros(E + 1, dtype=torch.int32, device="cuda")      # as many slots as x rows, all on one expert
    x = ops.Quantized(kind, q.x.codes.expand(300, -1).contiguous(), q.x.scales.expand(300, -1).contiguous(), K)
    many[e + 1:] = 300
    out = ops.expert_matmul(x, w, ws.view(-1), expert_start=many, out=F32)
    assert (out == out[0]).all()
    q.check(out[:1])


def test_products_on_two_streams_at_once(ops):
    """Each block takes a whole SM's tensor memory; two products that overlap share the SMs in turn."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    p = Problem(ops, ops.NVFP4, [70] * 30, 512, 640, seed=18)
    q = Problem(ops, ops.MXFP8, [1], 2048, 5120, seed=19)          # a cluster a tile
    want_p, want_q = p.run(out=F32), q.run(out=F32)
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        outs.append((p.run(out=F32, stream=a), q.run(out=F32, stream=b)))
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x, want_p) and torch.equal(y, want_q)
    assert ops.errors() == 0


# ---- activations over the range of float32 ---------------------------------------------------------------------------
# x codes of 0 make p = bias exactly, so the bias chooses the activation's argument.

def through_bias(ops, v, act, up_half=None, out=F32, **kw):
    """act(v), or act(v) * up_half gated, as the product's epilogue computes it for a 1-D v (a multiple of 128)."""
    N = v.numel() * (1 if up_half is None else 2)
    bias = v if up_half is None else torch.cat([v, up_half])
    x = ops.Quantized(ops.NVFP4, torch.zeros(1, 16, dtype=torch.uint8, device="cuda"),
                      torch.zeros(1, 16, dtype=torch.uint8, device="cuda"), 32)
    w = torch.zeros(1, N, 16, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(up(N, 128) * 4, dtype=torch.uint8, device="cuda")
    return ops.expert_matmul(x, w, ws, bias=bias.view(1, N), activation=act, gated=up_half is not None, out=out, **kw)


def activation(v, act):
    """The definition in 64 bits, and the argument of its sigmoid."""
    z = v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    return v / (1 + torch.exp(-z)), z


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_of_large_negative_sums_is_zero(ops, act):
    low = torch.finfo(BF16).min
    v = torch.tensor([-torch.finfo(F32).max, low, -1e38, -1e37, -1e35, -1e30, -1e20, -1e10, -1e5, -300.0] + [0.0] * 118, device="cuda")
    assert (through_bias(ops, v, act)[0] == 0).all()
    half = through_bias(ops, v.to(BF16), act, out=BF16)[0]                # the first is an infinity in bfloat16
    assert torch.isnan(half[0]) and (half[1:] == 0).all()
    big = torch.full_like(v, 1e30)
    assert (through_bias(ops, v, act, up_half=big)[0] == 0).all()
    # and large positive ones are themselves
    assert torch.equal(through_bias(ops, -v, act)[0], -v)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_relative_error(ops, act):
    """The exponential is within 2^-22, its sum with 1 and the quotient within 2^-23 each: 2^-20 in all.  GELU's
    argument z takes seven roundings of 2^-24 first, which the exponential turns into |z| 2^-21.  Below z = -86 two
    exponentials multiply, the second's argument of up to 150 rounded once: 2^-16, and the spacing of the smallest
    numbers."""
    g = gen(31)
    at = torch.cat([torch.linspace(-110, 30, 6000, device="cuda"), 4 * torch.randn(2048, device="cuda", generator=g),
                    torch.randn(144, device="cuda", generator=g) * 1e-3])
    got = through_bias(ops, at, act)[0].double()
    want, z = activation(at.double(), act)
    rel = 2.0 ** -20 + (z.abs() * 2.0 ** -21 if act == "gelu" else 0)
    rel = torch.where(z < -86, rel + 2.0 ** -16, rel)
    assert ((got - want).abs() <= rel * want.abs() + 2.0 ** -148).all()


# ---- codes of values far past what they can hold -----------------------------------------------------------------------

@pytest.mark.parametrize("g", [1e-3, 1e-10, 1e-30, 1.0])
def test_nvfp4_codes_saturate_with_their_sign(ops, g):
    """The quotient of a huge value and a small tensor scale passes float32's range: still 6 with the value's sign, and
    the block's other codes are the nearest ones."""
    top = torch.finfo(F32).max
    ts = torch.tensor([g], device="cuda")
    v = torch.zeros(128, device="cuda")
    v[0], v[1], v[17], v[18], v[33], v[50] = top, -top, -top, 4.8 * 448 * g, 1e35, torch.finfo(BF16).min
    v[34:40] = torch.tensor([0.3, -0.8, 1.3, -1.7, 2.6, -4.9], device="cuda") * 448 * g
    q = through_bias(ops, v, None, out=ops.NVFP4, out_tensor_scale=ts)
    c = code_values(q, ops)[0]
    s = scale_values(q.scales[:, :8], ops.NVFP4, ops)[0].repeat_interleave(16) * ts.double()
    want = torch.where(s > 0, v.double() / s, torch.zeros_like(s)).clamp(-6, 6)
    grid = torch.tensor(sorted(set(E2M1 + tuple(-e for e in E2M1))), dtype=torch.float64, device="cuda")
    assert torch.equal(c, grid[(want[:, None] - grid).abs().argmin(1)])
    # the norm's codes too: 128 equal values have norm 1, the weight makes them anything
    qn, _ = ops.rms_norm(torch.ones(1, 128, device="cuda"), v, ops.NVFP4, eps=0.0, tensor_scale=ts)
    assert torch.equal(code_values(qn, ops), code_values(q, ops)) and torch.equal(qn.scales[:, :8], q.scales[:, :8])


# ---- more columns than 31 bits of bytes ----------------------------------------------------------------------------------

def test_matmul_of_rows_past_2_31_bytes(ops):
    """Two float32 rows of 2^29 + 128 columns: the last block of columns starts 2^31 bytes into its row."""
    far, S = 1 << 29, 2
    q = Problem(ops, ops.NVFP4, [S], 256, 32, seed=24)
    w = torch.zeros(1, far + 128, 16, dtype=torch.uint8, device="cuda")
    ws = torch.zeros((far + 128) * 4, dtype=torch.uint8, device="cuda")       # a 128-row block is 512 bytes
    w[0, :128], w[0, far:] = q.w[0, :128], q.w[0, 128:]
    ws[:512], ws[-512:] = q.ws[:512], q.ws[512:]
    out = torch.full((S, far + 128), 5.0, device="cuda")
    ops.expert_matmul(q.x, w, ws, out=out)
    q.check(torch.cat([out[:, :128], out[:, far:]], 1))
    assert not out[:, 128:far].any()


# ---- the most tokens that a router call takes ---------------------------------------------------------------------------

def test_route_of_2_31_minus_1_tokens(ops):
    """One expert, k = 1: choice and slot of token t are 0 and t, except where the expert is off."""
    T = 2 ** 31 - 1
    v = torch.zeros(T, 1, dtype=BF16, device="cuda")
    v[5], v[T - 2] = -math.inf, -math.inf
    r = ops.route(v, 1)
    assert r.expert_start.tolist() == [0, T - 2]
    for lo in range(0, T, 1 << 28):
        hi = min(T, lo + (1 << 28))
        t = torch.arange(lo, hi, dtype=torch.int32, device="cuda")
        on = (t != 5) & (t != T - 2)
        assert torch.equal(r.ids[lo:hi, 0], on.int() - 1)
        assert torch.equal(r.weights[lo:hi, 0], on.float())
        slot = t - (t > 5).int() - (t > T - 2).int()
        assert torch.equal(r.slots[lo:hi, 0], torch.where(on, slot, torch.full_like(slot, -1)))
        row = t + (t >= 5).int() + (t >= T - 3).int()
        assert torch.equal(r.rows[lo:hi], torch.where(t < T - 2, row, torch.full_like(row, -1)))


# ---- rows whose squares leave float32's range ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("cols", [40, 64, 257, 1600, 5120, 5121, 20000])
def test_norm_of_rows_whose_squares_overflow_or_underflow(ops, cols, kind, dtype):
    g = gen(cols)
    x = torch.randn(6, cols, device="cuda", generator=g)
    size = torch.tensor([1e37, 1e25, 3e19, 1.0, 1e-25, 1e-37], device="cuda")[:, None]
    x = (x * size).to(dtype)
    x[0, 0] = torch.finfo(dtype).max
    w = (1 + 0.3 * torch.randn(cols, device="cuda", generator=g)).to(dtype)
    ts = torch.tensor([0.02], device="cuda") if kind == ops.NVFP4 else None
    q, _ = ops.rms_norm(x, w, kind, eps=0.0, tensor_scale=ts)
    check_norm(q, None, x, w, None, 0.0, ops)
    r = torch.zeros_like(x)
    q2, total = ops.rms_norm(x, w, kind, residual=r, eps=1e-6, tensor_scale=ts)
    check_norm(q2, total, x, w, r, 1e-6, ops)


@pytest.mark.parametrize("kind", [0, 1])
def test_norm_of_one_huge_value(ops, kind):
    """The row that test_norm_zero_huge_and_non_finite_rows makes: one value of 3e37 among 63 zeros has norm 8."""
    x = torch.zeros(2, 64, device="cuda")
    x[0, 5], x[1, 3] = 3e37, 1e-30
    w = torch.ones(64, device="cuda")
    q, _ = ops.rms_norm(x, w, kind, eps=1e-6)
    check_norm(q, None, x, w, None, 1e-6, ops)
    assert (values(q, ops)[0, 5] - 8).abs() <= 0.5 and (values(q, ops)[0].abs().sum() - 8).abs() <= 0.5


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("cols,off", [(64, 0), (64, 1), (640, 0), (4096, 0), (16400, 0)])
def test_norm_of_many_rows_some_out_of_range(ops, cols, off, kind):
    """Blocks that take several rows, the residual stream updated in place; a NaN weight of either sign marks nothing."""
    rows = 3000
    g = gen(cols + off)
    x = torch.randn(rows, cols, device="cuda", generator=g)
    r = torch.randn(rows, cols + off, device="cuda", generator=g)
    size = torch.ones(rows, 1, device="cuda")
    size[::5], size[3::7], size[2::11] = 1e30, 1e-30, 1e19
    x = (x * size).to(BF16)
    r = (r * size).to(BF16)[:, off:]
    w = (1 + 0.3 * torch.randn(cols, device="cuda", generator=g)).to(BF16)
    ts = torch.tensor([0.02], device="cuda") if kind == ops.NVFP4 else None
    r0, r1 = r.clone(), r.clone()
    q, total = ops.rms_norm(x, w, kind, residual=r, sum_out=r, eps=0.0, tensor_scale=ts)
    check_norm(q, total, x, w, r0, 0.0, ops)
    for sign in (-32768, 0):
        w2 = w.clone()
        w2.view(torch.int16)[0] = 0x7FC0 + sign
        r2 = r1.clone()
        q2, total2 = ops.rms_norm(x, w2, kind, residual=r2, sum_out=r2, eps=0.0, tensor_scale=ts)
        assert torch.equal(total2, total) and torch.equal(q2.scales[:, 1:], q.scales[:, 1:])
        block = 16 if kind == ops.NVFP4 else 32
        assert torch.isnan(scale_values(q2.scales[:, 0], kind, ops)).all()
        assert torch.equal(code_values(q2, ops)[:, block:], code_values(q, ops)[:, block:])


# ---- tensor scales of quantised outputs ---------------------------------------------------------------------------------

def test_a_quantized_output_brings_its_tensor_scale(ops):
    ts = torch.tensor([0.25], device="cuda")
    q = Problem(ops, ops.NVFP4, [9], 64, 64, seed=22)
    want = q.run(out=ops.NVFP4, out_tensor_scale=ts)
    mine = q.run(out=ops.empty_quantized(ops.NVFP4, 9, 64, tensor_scale=ts))
    assert mine.tensor_scale is ts
    assert torch.equal(mine.codes, want.codes) and torch.equal(mine.scales, want.scales)
    x, w = torch.randn(5, 64, **q.dev), torch.ones(64, device="cuda")
    want, _ = ops.rms_norm(x, w, ops.NVFP4, tensor_scale=ts)
    mine, _ = ops.rms_norm(x, w, ops.NVFP4, out=ops.empty_quantized(ops.NVFP4, 5, 64, tensor_scale=ts))
    assert mine.tensor_scale is ts
    assert torch.equal(mine.codes, want.codes) and torch.equal(mine.scales, want.scales)
    with pytest.raises(ops.CsfError, match="tensor scale"):
        q.run(out=ops.MXFP8, out_tensor_scale=ts)
    out = ops.empty_quantized(ops.MXFP8, 9, 64)
    with pytest.raises(ops.CsfError, match="tensor scale"):
        q.run(out=out, out_tensor_scale=ts)
    assert out.tensor_scale is None                       # a refused call changes nothing


# ---- streams and error words --------------------------------------------------------------------------------------------

def test_inputs_freed_while_another_stream_still_reads_them(ops):
    """A call on a side stream keeps what it reads until it has run, also where the caller lets go of it at once."""
    side = torch.cuda.Stream()
    q = Problem(ops, ops.NVFP4, [300], 256, 320, seed=23)
    w = torch.ones(1600, device="cuda")
    x, logits = torch.randn(3000, 1600, **q.dev), torch.randn(3000, 256, **q.dev)
    want_x, _ = ops.rms_norm(x, w, ops.MXFP8)
    want_r, want_p = ops.route(logits, 4), q.run(out=F32)
    torch.cuda.synchronize()
    x2, l2, p2 = x.clone(), logits.clone(), ops.Quantized(q.kind, q.x.codes.clone(), q.x.scales.clone(), q.K)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                     # some milliseconds
    got_x, _ = ops.rms_norm(x2, w, ops.MXFP8, stream=side)
    got_r = ops.route(l2, 4, stream=side)
    got_p = ops.expert_matmul(p2, q.w, q.ws, expert_start=q.start, out=F32, stream=side)
    shapes = [(t.shape, t.dtype) for t in (x2, l2, p2.codes, p2.scales)]
    del x2, l2, p2
    again = [torch.zeros(s, dtype=d, device="cuda") for s, d in shapes]      # would take the freed memory
    torch.cuda.synchronize()
    assert torch.equal(got_x.codes, want_x.codes) and torch.equal(got_p, want_p)
    assert torch.equal(got_r.ids, want_r.ids) and torch.equal(got_r.weights, want_r.weights)
    del again


def test_errors_of_a_captured_call_without_an_error_word(ops):
    """A call is captured with the device's own word or refused; replays report there."""
    from lossless_nvfp4_scale_gb300 import csf
    q = Problem(ops, ops.NVFP4, [6, 7], 64, 64, seed=8, gather=5)
    side = torch.cuda.Stream()
    out = torch.empty(13, 64, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q.run(out=out, error_word=torch.zeros(1, dtype=torch.int32, device="cuda"))       # no word of its own needed
    side.synchronize()
    kept = dict(ops._error_words)
    ops._error_words.clear()
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            with pytest.raises(ops.CsfError, match="capture"):
                q.run(out=out)
            q.run(out=out, error_word=torch.zeros(1, dtype=torch.int32, device="cuda"))
    finally:
        ops._error_words.clear()
        ops._error_words.update(kept)
    assert ops.errors() == 0                               # makes the word where there is none
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        q.run(out=out)
    graph.replay()
    assert ops.errors() == 0
    q.rows[2] = 99
    graph.replay()
    assert ops.errors() == csf.DEV_ERR_CORRUPT and ops.errors() == 0


def test_errors_of_two_threads_are_not_lost(ops):
    """One thread makes bad calls, another reads and clears: each bad call is seen by one that ends after it."""
    import threading
    from lossless_nvfp4_scale_gb300 import csf
    q = Problem(ops, ops.NVFP4, [6, 7], 64, 64, seed=8, gather=5)
    q.rows[2] = 99
    ops.errors()
    stop, seen, side = threading.Event(), [], torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def reader():
        while not stop.is_set():
            seen.append(ops.errors())
    t = threading.Thread(target=reader)
    t.start()
    lost = 0
    try:
        for _ in range(300):
            before = len(seen)
            q.run(stream=side)
            side.synchronize()
            ended = len(seen)
            while len(seen) < ended + 2:                   # the second of these began after the call had ended
                pass
            lost += csf.DEV_ERR_CORRUPT not in seen[before:]
    finally:
        stop.set()
        t.join()
    assert lost == 0
