"""Measured cases of the expert-layer operators: the norm that quantises a layer's input, the experts' block-scaled
products with their epilogues, and the router that groups tokens by expert.

`run` computes an operator either with the library's kernels (`own`) or in its plain form, elementary torch operations
in 32 bits.  `exact` states each operator's definition in 64 bits.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"mxfp8": 32, "nvfp4": 16}     # elements that share a scale
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # The norm before one decoded token's experts, with the residual stream's addition: the latency of one call.
        dict(name="norm_token", op="norm", tokens=1, cols=1600, kind="nvfp4", dtype="bf16", residual=True),
        # A decode batch whose width is no multiple of a block: padded columns, a ragged last block.
        dict(name="norm_ragged", op="norm", tokens=777, cols=1001, kind="nvfp4", dtype="f32", residual=False),
        # A long prompt in a wide model: the bandwidth of the largest call.
        dict(name="norm_prompt", op="norm", tokens=16384, cols=5120, kind="mxfp8", dtype="bf16", residual=True),
        # One decoded token through one dense block-scaled projection with a bias.
        dict(name="matmul_token", op="matmul", kind="mxfp8", experts=1, slots=1, rows=2048, cols=5120, active=1,
             act="none", gated=False, bias=True, residual=False, gather=False, out="bf16"),
        # A small decode batch: 64 routed slots on 8 of the 512 gate/up experts, SwiGLU in the epilogue.
        dict(name="matmul_routed", op="matmul", kind="nvfp4", experts=512, slots=64, rows=1024, cols=1600, active=8,
             act="silu", gated=True, bias=False, residual=False, gather=True, out="bf16"),
        # A prompt of 4096 tokens, 8 experts each, through the 512 fused gate/up experts.
        dict(name="matmul_gate", op="matmul", kind="nvfp4", experts=512, slots=32768, rows=1024, cols=1600, active=512,
             act="silu", gated=True, bias=False, residual=False, gather=True, out="bf16"),
        # The same prompt through the down experts, the rows weighted and added to a residual.
        dict(name="matmul_down", op="matmul", kind="nvfp4", experts=512, slots=32768, rows=2048, cols=800, active=512,
             act="none", gated=False, bias=True, residual=True, gather=False, out="bf16"),
        # A batch of 500 tokens, 4 experts each, through 384 MXFP4 experts; the next product's 8-bit input comes out.
        dict(name="matmul_mxfp4", op="matmul", kind="mxfp8", experts=384, slots=2000, rows=2048, cols=5120, active=384,
             act="silu", gated=True, bias=False, residual=False, gather=True, out="mxfp8"),
        # A long prompt through one dense projection: bound by the matrix instructions.
        dict(name="matmul_prompt", op="matmul", kind="mxfp8", experts=1, slots=8191, rows=2048, cols=5120, active=1,
             act="gelu", gated=False, bias=True, residual=True, gather=False, out="bf16"),
        # The router of one decoded token.
        dict(name="route_token", op="route", tokens=1, experts=512, k=8, dtype="f32", masked=False, renormalize=True),
        # A decode batch over an odd number of experts, some of them switched off.
        dict(name="route_masked", op="route", tokens=333, experts=129, k=6, dtype="f32", masked=True, renormalize=False),
        # The router of a long prompt.
        dict(name="route_prompt", op="route", tokens=32768, experts=384, k=8, dtype="bf16", masked=False,
             renormalize=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "matmul", "matmul", "route"])
    if op == "norm":
        return dict(op=op, tokens=_spread(rng, 1, 16384), cols=_spread(rng, 33, 5120), kind=rng.choice(["mxfp8", "nvfp4"]),
                    dtype=rng.choice(["bf16", "f16", "f32"]), residual=rng.random() < 0.6)
    if op == "route":
        experts = _spread(rng, 8, 1024)
        return dict(op=op, tokens=_spread(rng, 1, 16384), experts=experts, k=rng.randint(1, 8),
                    dtype=rng.choice(["bf16", "f32"]), masked=rng.random() < 0.3, renormalize=rng.random() < 0.5)
    kind = rng.choice(["mxfp8", "nvfp4"])
    gated = rng.random() < 0.5
    experts = 1 if rng.random() < 0.3 else _spread(rng, 2, 512)
    cols = 128 * _spread(rng, 1, 40) if kind == "mxfp8" else 32 * _spread(rng, 2, 100)
    rows = 256 * rng.randint(1, 8) if gated else _spread(rng, 64, 2048)
    if experts > 1:
        experts = max(2, min(experts, int(3.5e9 / (rows * cols))))
    slots = _spread(rng, 1, 32768)
    slots = max(1, min(slots, int(5e10 / (rows * cols))))
    return dict(op=op, kind=kind, experts=experts, slots=slots, rows=rows, cols=cols,
                active=max(1, min(experts, slots, _spread(rng, max(1, experts // 16), experts))),
                act="silu" if gated else rng.choice(["none", "relu", "gelu", "silu"]), gated=gated,
                bias=rng.random() < 0.5, residual=not gated and rng.random() < 0.5,
                gather=experts > 1 and rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "f32", kind]))


# ---- inputs ----------------------------------------------------------------------------------------------------------

def _up(n, m):
    return -(-n // m) * m


def _blocked(scales):
    """[E, N, C] scale bytes in the 128 x 4 tiled scale-operand layout, flat, padding 0."""
    E, N, C = scales.shape
    p = torch.zeros(E, _up(N, 128), _up(C, 4), dtype=torch.uint8, device=scales.device)
    p[:, :N, :C] = scales
    p = p.view(E, -1, 4, 32, p.shape[2] // 4, 4)          # row block, a, b, column block, c
    return p.permute(0, 1, 4, 3, 2, 5).reshape(-1)


def _scale_bytes(g, kind, shape):
    """Scale bytes as quantised tensors hold them: UE4M3 around 0.1, or UE8M0 around 2^-4."""
    lo, hi = (0x14, 0x2c) if kind == "nvfp4" else (120, 126)
    return torch.randint(lo, hi, shape, dtype=torch.uint8, device="cuda", generator=g)


def _codes(g, kind, shape):
    """Code bytes: two E2M1 values each, or an E4M3 value of small magnitude."""
    b = torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)
    if kind == "mxfp8":
        b = (b & 0x80) | (0x20 + (b & 0x7F) % 0x30)       # +-2^-3 .. 7.5, no NaN
    return b


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    if case["op"] == "norm":
        T, H, dt = case["tokens"], case["cols"], DTYPES[case["dtype"]]
        x = (rand(T, H) * (0.5 + rand(T, 1).abs())).to(dt)
        return dict(case=case, x=x, weight=(1 + 0.2 * rand(H)).to(dt), residual=rand(T, H).to(dt) if case["residual"] else None,
                    tensor_scale=torch.full((1,), 0.01, device="cuda") if case["kind"] == "nvfp4" else None)
    if case["op"] == "route":
        T, E = case["tokens"], case["experts"]
        logits = 1.5 * rand(T, E)
        if case["masked"]:                                # experts switched off, and rows with few or none left
            logits[torch.rand(T, E, device="cuda", generator=g) < 0.2] = -math.inf
            logits[1::7, 2:] = -math.inf
            logits[3::50] = -math.inf
        return dict(case=case, logits=logits.to(DTYPES[case["dtype"]]))
    kind, E, S, N, K = case["kind"], case["experts"], case["slots"], case["rows"], case["cols"]
    F, B = N // 2 if case["gated"] else N, BLOCK[case["kind"]]
    T = max(1, S // 4) if case["gather"] else S
    # routing: `active` experts share the slots, each one at least
    ids = torch.randperm(E, device="cuda", generator=g)[:case["active"]]
    extra = torch.randint(0, case["active"], (S - case["active"],), device="cuda", generator=g)
    ids = torch.cat([ids, ids[extra]])
    counts = torch.bincount(ids, minlength=E)
    start = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    start[1:] = counts.cumsum(0)
    scales = torch.zeros(T, _up(K // B, 16), dtype=torch.uint8, device="cuda")
    scales[:, :K // B] = _scale_bytes(g, kind, (T, K // B))
    C = K // BLOCK["mxfp8"] if kind == "mxfp8" else K // BLOCK["nvfp4"]
    return dict(
        case=case, most=int(counts.max()),
        x=_codes(g, kind, (T, K if kind == "mxfp8" else K // 2)), x_scales=scales,
        w=_codes(g, "nvfp4", (E, N, K // 2)), w_scales=_blocked(_scale_bytes(g, kind, (E, N, C))),
        start=start if E > 1 else None,
        index=torch.randint(0, T, (S,), dtype=torch.int32, device="cuda", generator=g) if case["gather"] else None,
        alpha=0.5 + torch.rand(E, device="cuda", generator=g),
        bias=rand(E, N).to(torch.bfloat16) if case["bias"] else None,
        row_scale=torch.rand(S, device="cuda", generator=g) if case["residual"] else None,
        residual=rand(S, F).to(torch.bfloat16) if case["residual"] else None,
        out_scale=torch.full((1,), 0.05, device="cuda") if case["out"] == "nvfp4" else None)


# ---- the plain form --------------------------------------------------------------------------------------------------

def _to_e2m1(v):
    """Nearest E2M1 value, ties to even, saturating."""
    a = v.abs()
    r = (0.5 * ((a > 0.25).to(v.dtype) + (a >= 0.75) + (a > 1.25).to(v.dtype) + (a >= 1.75))
         + (a > 2.5).to(v.dtype) + (a >= 3.5) + 2.0 * (a > 5).to(v.dtype))
    return torch.where(v < 0, -r, r)


def _quantize(y, kind, tensor_scale):
    """The codes and scales of y's rows as the values they stand for, columns padded to a multiple of 32 with zeros."""
    rows, cols = y.shape
    y = torch.nn.functional.pad(y, (0, _up(cols, 32) - cols)).view(rows, -1, BLOCK[kind])
    amax = y.abs().amax(2)
    if kind == "mxfp8":       # the smallest power of two that keeps the block's values within 448
        m, e = torch.frexp(amax)
        e = torch.where(amax > 0, e - 9 + (m > 0.875), torch.full_like(e, -127)).clamp(-127, 127)
        q = torch.ldexp(y, -e[..., None])
        scale = torch.ldexp(torch.ones_like(amax), e)
        return q.view(rows, -1).to(torch.float8_e4m3fn), scale.to(torch.float8_e8m0fnu)
    scale = (amax / (6 * tensor_scale)).clamp(max=448).to(torch.float8_e4m3fn)
    whole = (scale.to(y.dtype) * tensor_scale)[..., None]
    q = torch.where(whole > 0, y / whole, torch.zeros_like(y))
    return _to_e2m1(q).view(rows, -1).to(torch.float8_e4m3fn), scale


def _unpack(codes):
    """Packed E2M1 codes as values, in 32 bits."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    return torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)


def _scale_values(b, kind):
    return b.view(torch.float8_e4m3fn).float() if kind == "nvfp4" else torch.ldexp(torch.ones((), device=b.device), b.int() - 127)


def _weights(s, experts=slice(None), to=torch.float32):
    """The weights of some experts as values: [E, N, K]."""
    c = s["case"]
    E, N, K, B = c["experts"], c["rows"], c["cols"], BLOCK[c["kind"]]
    sc = s["w_scales"].view(E, _up(N, 128) // 128, -1, 32, 4, 4)[experts].permute(0, 1, 4, 3, 2, 5)
    sc = sc.reshape(sc.shape[0], _up(N, 128), -1)[:, :N, :K // B]
    v = _unpack(s["w"][experts]).to(to).view(-1, N, K // B, B)
    return v.mul_(_scale_values(sc, c["kind"]).to(to)[..., None]).view(-1, N, K)


def _inputs(s, to=torch.float32):
    """The quantised rows as values: [T, K]."""
    c = s["case"]
    K, B = c["cols"], BLOCK[c["kind"]]
    v = s["x"].view(torch.float8_e4m3fn).to(to) if c["kind"] == "mxfp8" else _unpack(s["x"]).to(to)
    return (v.view(v.shape[0], -1, B) * _scale_values(s["x_scales"][:, :K // B], c["kind"]).to(to)[..., None]).view(-1, K)


def _act(v, name):
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":        # the tanh form
        return v / (1 + torch.exp(-1.5957691216057308 * (v + 0.044715 * v * v * v)))
    return v.clamp(min=0) if name == "relu" else v


def _epilogue(s, y, e):
    """The epilogue on products y [S, N] of slots whose experts are e, in y's type."""
    c, to = s["case"], y.dtype
    y = y * s["alpha"].to(to)[e][:, None]
    if s["bias"] is not None:
        y = y + s["bias"].to(to)[e]
    if c["gated"]:
        half = c["rows"] // 2
        y = _act(y[:, :half], c["act"]) * y[:, half:]
    else:
        y = _act(y, c["act"])
    if s["residual"] is not None:
        y = y * s["row_scale"].to(to)[:, None] + s["residual"].to(to)
    return y


def _plain_matmul(s):
    c = s["case"]
    S, E, dev = c["slots"], c["experts"], s["x"].device
    x, w = _inputs(s), _weights(s)
    slot = torch.arange(S, device=dev)
    start = s["start"].long() if s["start"] is not None else torch.tensor([0, S], device=dev)
    e = torch.searchsorted(start[1:], slot, right=True)
    at = (start[:-1, None] + torch.arange(s["most"], device=dev)).clamp(max=S - 1)      # [E, most] slots, padded
    rows = s["index"].long()[at] if s["index"] is not None else at
    y = torch.bmm(x[rows.view(-1)].view(E, s["most"], -1), w.transpose(1, 2))
    y = _epilogue(s, y[e, slot - start[e]], e)
    if c["out"] in BLOCK:
        return dict(zip(("codes", "scales"), _quantize(y, c["out"], s["out_scale"])))
    return y.to(DTYPES[c["out"]])


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["weight"].float()
    codes, scales = _quantize(y, c["kind"], s["tensor_scale"])
    return dict(codes=codes, scales=scales, sum=h.to(s["x"].dtype) if s["residual"] is not None else None)


def _plain_route(s):
    c = s["case"]
    E, k, T = c["experts"], c["k"], c["tokens"]
    v = s["logits"].float()
    order = torch.sort(v, dim=1, descending=True, stable=True)        # ties to the lowest expert
    top, ids = order.values[:, :k], order.indices[:, :k]
    on = top > -math.inf
    p = torch.where(on, torch.exp(top - top[:, :1]), torch.zeros_like(top))
    total = p.sum(1, keepdim=True) if c["renormalize"] else torch.exp(v - top[:, :1]).sum(1, keepdim=True)
    weights = torch.where(on, p / total, torch.zeros_like(p))
    flat = torch.where(on, ids, torch.full_like(ids, E)).reshape(-1)
    start = torch.searchsorted(flat.sort().values, torch.arange(E + 1, device=v.device))
    slot_of = torch.argsort(flat, stable=True)                        # slots: by expert, then by token
    slots = torch.empty_like(flat)
    slots[slot_of] = torch.arange(T * k, device=v.device)
    used = torch.arange(T * k, device=v.device) < start[E]
    rows = torch.where(used, slot_of // k, torch.full_like(slot_of, -1))
    return dict(ids=torch.where(on, ids, torch.full_like(ids, -1)).int(), weights=weights, start=start.int(), rows=rows.int(),
                slots=torch.where(on.reshape(-1), slots, torch.full_like(slots, -1)).view(T, k).int())


# ---- the library's kernels -------------------------------------------------------------------------------------------

def _as_values(q, ops):
    """A quantised result's codes and scales in the types of the values they stand for."""
    if q.kind == ops.MXFP8:
        return q.codes.view(torch.float8_e4m3fn), q.scales[:, :q.codes.shape[1] // 32].view(torch.float8_e8m0fnu)
    table = _E4M3_PAIRS.get(q.codes.device)
    if table is None:         # the two E2M1 codes of a byte as two E4M3 bytes
        one = torch.tensor(E2M1 + tuple(-v for v in E2M1)).to(torch.float8_e4m3fn).view(torch.uint8).int()
        b = torch.arange(256)
        pairs = (one[b & 15] | (one[b >> 4] << 8)).to(torch.int32)
        table = _E4M3_PAIRS[q.codes.device] = torch.where(pairs > 32767, pairs - 65536, pairs).to(torch.int16).to(q.codes.device)
    values = table[q.codes.int()].view(torch.uint8).view(torch.float8_e4m3fn)
    return values, q.scales[:, :q.codes.shape[1] // 8].view(torch.float8_e4m3fn)


_E4M3_PAIRS = {}              # constant tables, one a device


def _own(s):
    from lossless_nvfp4_scale_gb300 import ops
    c = s["case"]
    kind = {"mxfp8": ops.MXFP8, "nvfp4": ops.NVFP4}
    if c["op"] == "norm":
        q, total = ops.rms_norm(s["x"], s["weight"], kind[c["kind"]], residual=s["residual"], eps=EPS,
                                tensor_scale=s["tensor_scale"])
        codes, scales = _as_values(q, ops)
        return dict(codes=codes, scales=scales, sum=total)
    if c["op"] == "route":
        r = ops.route(s["logits"], c["k"], renormalize=c["renormalize"])
        return dict(ids=r.ids, weights=r.weights, start=r.expert_start, rows=r.rows, slots=r.slots)
    out = kind[c["out"]] if c["out"] in kind else DTYPES[c["out"]]
    y = ops.expert_matmul(ops.Quantized(kind[c["kind"]], s["x"], s["x_scales"], c["cols"]), s["w"], s["w_scales"],
                          expert_start=s["start"], rows=s["index"], alpha=s["alpha"], bias=s["bias"],
                          activation=c["act"], gated=c["gated"], row_scale=s["row_scale"], residual=s["residual"],
                          out=out, out_tensor_scale=s["out_scale"])
    return dict(zip(("codes", "scales"), _as_values(y, ops))) if c["out"] in BLOCK else y


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "matmul": _plain_matmul, "route": _plain_route}[state["case"]["op"]](state)


# ---- work and the definition in 64 bits ------------------------------------------------------------------------------

def _coded(kind, n, cols):
    """Bytes of n rows of codes and scales."""
    cols = _up(cols, 32)
    return n * (cols + cols // 32 if kind == "mxfp8" else cols // 2 + cols // 16)


def work(case):
    if case["op"] == "norm":
        size = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
        T, H = case["tokens"], case["cols"]
        return {"bytes": T * H * size * (3 if case["residual"] else 1) + H * size + _coded(case["kind"], T, H), "flops": 6 * T * H}
    if case["op"] == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        return {"bytes": T * E * (2 if case["dtype"] == "bf16" else 4) + 4 * (4 * T * k + E + 1), "flops": 4 * T * E}
    E, S, N, K = case["active"], case["slots"], case["rows"], case["cols"]
    F = N // 2 if case["gated"] else N
    T = max(1, S // 4) if case["gather"] else S
    weights = E * N * (K // 2 + K // (32 if case["kind"] == "mxfp8" else 16))
    out = _coded(case["out"], S, F) if case["out"] in BLOCK else S * F * (4 if case["out"] == "f32" else 2)
    return {"bytes": weights + _coded(case["kind"], T, K) + out + (2 * E * N if case["bias"] else 0)
            + (S * (2 * F + 4) if case["residual"] else 0) + (4 * S if case["gather"] else 0), "flops": 2 * S * N * K}


def _exact_quantize(y, kind, tensor_scale):
    rows, cols = y.shape
    y = torch.nn.functional.pad(y, (0, _up(cols, 32) - cols)).view(rows, -1, BLOCK[kind])
    amax = y.abs().amax(2)
    if kind == "mxfp8":
        e = torch.ceil(torch.log2((amax / 448).clamp(min=2.0 ** -127)))
        e = torch.where(amax > 448 * torch.exp2(e), e + 1, torch.where(amax <= 448 * torch.exp2(e - 1), e - 1, e)).clamp(-127, 127)
        scale = torch.exp2(e)
        return (y / scale[..., None]).to(torch.float8_e4m3fn).double().view(rows, -1), scale
    scale = (amax / (6 * tensor_scale.double())).clamp(max=448).to(torch.float8_e4m3fn).double()
    grid = torch.tensor(E2M1, dtype=torch.float64, device=y.device)
    v = torch.where(scale[..., None] > 0, y.abs() / (scale * tensor_scale.double())[..., None], torch.zeros_like(y)).clamp(max=6)
    up = torch.searchsorted(grid, v).clamp(max=7)
    low = (up - 1).clamp(min=0)
    d = (v - grid[low]) - (grid[up] - v)
    at = torch.where(d > 0, up, torch.where(d < 0, low, torch.where(low % 2 == 0, low, up)))
    at = torch.where(v == grid[up], up, at)
    return (torch.sign(y) * grid[at]).view(rows, -1), scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double() + (s["residual"].double() if s["residual"] is not None else 0)
        y = h / ((h * h).sum(1, keepdim=True) / case["cols"] + EPS).sqrt() * s["weight"].double()
        codes, scales = _exact_quantize(y, case["kind"], s["tensor_scale"])
        return dict(codes=codes, scales=scales, sum=h if s["residual"] is not None else None)
    if case["op"] == "route":
        v = s["logits"].double()
        ids = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :case["k"]]
        p = torch.nan_to_num(torch.softmax(v, 1)).gather(1, ids)
        if case["renormalize"]:
            p = torch.nan_to_num(p / p.sum(1, keepdim=True))
        return dict(ids=None, weights=p, start=None, rows=None, slots=None)
    f64, dev = torch.float64, s["x"].device
    S = case["slots"]
    start = s["start"].tolist() if s["start"] is not None else [0, S]
    x = _inputs(s, f64)
    x = x[s["index"].long()] if s["index"] is not None else x
    y = torch.zeros(S, case["rows"], dtype=f64, device=dev)
    for i in range(case["experts"]):
        lo, hi = start[i], start[i + 1]
        if hi > lo:
            y[lo:hi] = x[lo:hi] @ _weights(s, slice(i, i + 1), f64)[0].T
    e = torch.repeat_interleave(torch.arange(case["experts"], device=dev), torch.tensor(start, device=dev).diff())
    y = _epilogue(s, y, e)
    if case["out"] in BLOCK:
        return dict(zip(("codes", "scales"), _exact_quantize(y, case["out"], s["out_scale"])))
    return y
