"""Measured cases of the operators that carry an expert layer's 8-bit products and its tokens: the product with a scale
for each block of 128, the rows sent to their experts' slots (quantised on the way) and back with the router's weights,
and the gradients of that way and of the router.

`run` computes an operator either with the library's kernels (`own`) or in its plain form, elementary torch operations
in 32 bits.  `exact` states each operator's definition in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128                            # elements that share a scale
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # One decoded token through one dense 8-bit projection with a bias: the latency of one call.
        dict(name="matmul_token", op="matmul", experts=1, slots=1, rows=2048, cols=5120, active=1, transposed=False,
             act="none", gated=False, bias=True, residual=False, gather=False, out="bf16"),
        # A small decode batch: 64 routed slots on 8 of 128 gate/up experts whose depth is no multiple of a block.
        dict(name="matmul_routed", op="matmul", experts=128, slots=64, rows=1024, cols=1600, active=8, transposed=False,
             act="silu", gated=True, bias=False, residual=False, gather=True, out="bf16"),
        # A prompt of 4096 tokens, 8 experts each, through 128 gate/up experts; the down product's 8-bit input comes out.
        dict(name="matmul_experts", op="matmul", experts=128, slots=32768, rows=4096, cols=2048, active=128,
             transposed=False, act="silu", gated=True, bias=False, residual=False, gather=True, out="fp8"),
        # A long prompt through one dense projection, added to the residual stream: bound by the matrix instructions.
        dict(name="matmul_prompt", op="matmul", experts=1, slots=8191, rows=5120, cols=5120, active=1, transposed=False,
             act="none", gated=False, bias=False, residual=True, gather=False, out="bf16"),
        # The gradient of an expert product's input, 1000 tokens on 4 of 64 experts each: the weights the other way.
        dict(name="matmul_input_grad", op="matmul", experts=64, slots=4000, rows=1600, cols=2048, active=64,
             transposed=True, act="none", gated=False, bias=False, residual=False, gather=False, out="bf16"),
        # The quantiser before a dense product, of a batch whose width is no multiple of a block.
        dict(name="quantize_ragged", op="dispatch", tokens=777, cols=1001, k=0, dtype="f32", masked=False, out="fp8"),
        # A prompt's rows to their experts' slots, quantised once and written 8 times.
        dict(name="dispatch_prompt", op="dispatch", tokens=8192, cols=2048, k=8, dtype="bf16", masked=False, out="fp8"),
        # One decoded token's experts added up with the router's weights.
        dict(name="combine_token", op="combine", tokens=1, cols=5120, k=8, dtype="bf16", masked=False, residual=True),
        # The same for a prompt.
        dict(name="combine_prompt", op="combine", tokens=4095, cols=5120, k=8, dtype="bf16", masked=False, residual=True),
        # The gradient of that sum, for the experts' rows and the weights; tokens with fewer experts than k, or none.
        dict(name="combine_grad", op="combine_grad", tokens=3001, cols=1600, k=6, dtype="bf16", masked=True, out="bf16"),
        # The router's gradient for a few tokens that train beside others, renormalised weights.
        dict(name="route_grad_few", op="route_grad", tokens=33, experts=129, k=6, dtype="f32", masked=True, renormalize=True),
        # The router's gradient of a long prompt, weights of a softmax over all experts.
        dict(name="route_grad_prompt", op="route_grad", tokens=32768, experts=384, k=8, dtype="bf16", masked=False,
             renormalize=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul", "dispatch", "combine", "combine_grad", "route_grad"])
    if op == "route_grad":
        experts = _spread(rng, 8, 1024)
        return dict(op=op, tokens=_spread(rng, 1, 32768 * 384 // max(experts, 384)), experts=experts, k=rng.randint(1, 8),
                    dtype=rng.choice(["bf16", "f32"]), masked=rng.random() < 0.4, renormalize=rng.random() < 0.5)
    if op == "matmul":
        transposed = rng.random() < 0.25
        gated = not transposed and rng.random() < 0.5
        experts = 1 if rng.random() < 0.4 else _spread(rng, 2, 256)
        cols = 16 * _spread(rng, 4, 320)
        rows = 256 * rng.randint(1, 16) if gated else 16 * _spread(rng, 4, 320) if transposed else _spread(rng, 64, 5120)
        if experts > 1:
            experts = max(2, min(experts, int(6e8 / (rows * cols))))
        slots = max(1, min(_spread(rng, 1, 32768), int(2.1e11 / (rows * cols)), int(1.1e8 / cols)))
        return dict(op=op, experts=experts, slots=slots, rows=rows, cols=cols, transposed=transposed,
                    active=max(1, min(experts, slots, _spread(rng, max(1, experts // 16), experts))),
                    act="silu" if gated else "none" if transposed else rng.choice(["none", "relu", "gelu", "silu"]),
                    gated=gated, bias=not transposed and rng.random() < 0.5, residual=not gated and rng.random() < 0.4,
                    gather=experts > 1 and rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "f32", "fp8"]))
    cols, k = _spread(rng, 33, 5120), rng.randint(1, 8)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    tokens = _spread(rng, 1, min(8192, int(1.6e8 / (cols * k * SIZES[dtype] / 2))))
    if op == "dispatch":
        k = 0 if rng.random() < 0.3 else k
        return dict(op=op, tokens=tokens, cols=cols, k=k, dtype=dtype, masked=k > 0 and rng.random() < 0.3,
                    out=rng.choice(["fp8", "fp8", dtype]) if k else "fp8")
    masked = rng.random() < 0.3
    if op == "combine":
        return dict(op=op, tokens=tokens, cols=cols, k=k, dtype=dtype, masked=masked, residual=rng.random() < 0.5)
    return dict(op=op, tokens=max(1, tokens // 2), cols=cols, k=k, dtype=dtype, masked=masked, out=rng.choice(["fp8", dtype, dtype]))


# ---- inputs ----------------------------------------------------------------------------------------------------------

def _up(n, m):
    return -(-n // m) * m


def _blocks(n):
    return -(-n // BLOCK)


def _codes(g, *shape):
    """E4M3 values as quantised normal numbers have them: the largest of a block near 448."""
    return (torch.randn(*shape, device="cuda", generator=g) * 140).clamp_(-448, 448).to(torch.float8_e4m3fn)


def _routes(g, T, k, masked):
    """Slots of T tokens' k choices, sorted by an expert drawn at random; -1 where a choice fell away (`masked`): some
    tokens have one choice left, some none."""
    expert = torch.randint(0, 64, (T, k), device="cuda", generator=g)
    if masked:
        off = torch.rand(T, k, device="cuda", generator=g) < 0.2
        off[1::7, 1:] = True
        off[3::50] = True
        expert[off] = 64
    flat = expert.view(-1)
    slots = torch.empty(T * k, dtype=torch.int32, device="cuda")
    slots[torch.argsort(flat, stable=True)] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    return torch.where(flat < 64, slots, torch.full_like(slots, -1)).view(T, k)


def _empty_rows(rows, cols):
    """Zeroed codes and scales of FP8 rows: slots that no choice has keep them."""
    return (torch.zeros(rows, _up(cols, 32), dtype=torch.uint8, device="cuda"),
            torch.zeros(rows, _up(4 * _blocks(cols), 16), dtype=torch.uint8, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    if case["op"] == "route_grad":
        T, E, k = case["tokens"], case["experts"], case["k"]
        logits = 1.5 * rand(T, E)
        if case["masked"]:                                # experts switched off, and rows with few or none left
            logits[torch.rand(T, E, device="cuda", generator=g) < 0.2] = -math.inf
            logits[1::7, 2:] = -math.inf
            logits[3::50] = -math.inf
        logits = logits.to(DTYPES[case["dtype"]])
        top, ids = torch.sort(logits.float(), dim=1, descending=True, stable=True)
        on = top[:, :k] > -math.inf
        p = torch.nan_to_num(torch.softmax(logits.float(), 1)).gather(1, ids[:, :k])
        if case["renormalize"]:
            p = torch.nan_to_num(p / p.sum(1, keepdim=True))
        return dict(case=case, logits=logits, ids=torch.where(on, ids[:, :k], -1).int(),
                    weights=torch.where(on, p, torch.zeros_like(p)), dweights=rand(T, k))
    if case["op"] != "matmul":
        T, H, k, dt = case["tokens"], case["cols"], case["k"], DTYPES[case["dtype"]]
        s = dict(case=case, slots=_routes(g, T, k, case["masked"]) if k else None)
        if case["op"] == "dispatch":
            s["x"] = (rand(T, H) * (0.5 + rand(T, 1).abs())).to(dt)
        else:
            s["y"] = rand(T * k, H).to(dt)
            s["weights"] = torch.softmax(rand(T, k), 1).where(s["slots"] >= 0, torch.zeros((), device="cuda"))
            s["x"] = rand(T, H).to(dt) if case["op"] == "combine_grad" or case["residual"] else None
        if case["op"] != "combine":                       # where the slots' rows go
            S = T * k if k else T
            s["out"] = _empty_rows(S, H) if case["out"] == "fp8" else torch.zeros(S, H, dtype=dt, device="cuda")
        return s
    E, S, N, K = case["experts"], case["slots"], case["rows"], case["cols"]
    depth, F = (N, K) if case["transposed"] else (K, N // 2 if case["gated"] else N)
    T = max(1, S // 4) if case["gather"] else S
    # routing: `active` experts share the slots, each one at least
    ids = torch.randperm(E, device="cuda", generator=g)[:case["active"]]
    extra = torch.randint(0, case["active"], (S - case["active"],), device="cuda", generator=g)
    counts = torch.bincount(torch.cat([ids, ids[extra]]), minlength=E)
    start = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    start[1:] = counts.cumsum(0)
    scales = torch.zeros(T, _up(4 * _blocks(depth), 16) // 4, device="cuda")
    scales[:, :_blocks(depth)] = (0.5 + torch.rand(T, _blocks(depth), device="cuda", generator=g)) / 140
    return dict(
        case=case, most=int(counts.max()), chosen=ids.sort().values,
        x=torch.nn.functional.pad(_codes(g, T, depth).view(torch.uint8), (0, _up(depth, 32) - depth)),
        x_scales=scales.view(torch.uint8),
        w=_codes(g, E, N, K),
        w_scales=(0.5 + torch.rand(E, _blocks(N), _blocks(K), device="cuda", generator=g)) / (140 * depth ** 0.5),
        start=start if E > 1 else None,
        index=torch.randint(0, T, (S,), dtype=torch.int32, device="cuda", generator=g) if case["gather"] else None,
        bias=rand(E, N).to(torch.bfloat16) if case["bias"] else None,
        row_scale=torch.rand(S, device="cuda", generator=g) if case["residual"] else None,
        residual=rand(S, F).to(torch.bfloat16) if case["residual"] else None)


# ---- the plain form --------------------------------------------------------------------------------------------------

def _quantize(y):
    """FP8 codes and scales of y's rows, columns padded to a multiple of 32 with zeros."""
    rows, cols = y.shape
    v = torch.nn.functional.pad(y, (0, _up(cols, BLOCK) - cols)).view(rows, -1, BLOCK)
    scale = (v.abs().amax(2) / 448).clamp(min=2.0 ** -126)
    q = (v / scale[..., None]).to(torch.float8_e4m3fn).view(rows, -1)
    return q[:, :_up(cols, 32)].contiguous(), scale


def _weights(s, experts):
    """The weights of some experts as values: [E, N, K]."""
    w = s["w"][experts]
    E, N, K = w.shape
    scale = s["w_scales"][experts].repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]
    return w.float() * scale


def _inputs(s):
    """The quantised rows as values: [T, depth]."""
    c = s["case"]
    depth = c["rows"] if c["transposed"] else c["cols"]
    scale = s["x_scales"].view(torch.float32).repeat_interleave(BLOCK, 1)[:, :depth]
    return s["x"].view(torch.float8_e4m3fn)[:, :depth].float() * scale


def _act(v, name):
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":        # the tanh form
        return v / (1 + torch.exp(-1.5957691216057308 * (v + 0.044715 * v * v * v)))
    return v.clamp(min=0) if name == "relu" else v


def _epilogue(s, y, e):
    """The epilogue on products y [S, F] of slots whose experts are e."""
    c = s["case"]
    if s["bias"] is not None:
        y = y + s["bias"].float()[e]
    if c["gated"]:
        half = c["rows"] // 2
        y = _act(y[:, :half], c["act"]) * y[:, half:]
    else:
        y = _act(y, c["act"])
    if s["residual"] is not None:
        y = y * s["row_scale"][:, None] + s["residual"].float()
    return y


def _plain_matmul(s):
    c = s["case"]
    S, chosen, dev = c["slots"], s["chosen"], s["x"].device
    x, w = _inputs(s), _weights(s, chosen)
    slot = torch.arange(S, device=dev)
    start = s["start"].long() if s["start"] is not None else torch.tensor([0, S], device=dev)
    first = start[chosen]
    nth = torch.searchsorted(first, slot, right=True) - 1                                # a slot's expert among the chosen
    at = (first[:, None] + torch.arange(s["most"], device=dev)).clamp(max=S - 1)         # [chosen, most] slots, padded
    rows = s["index"].long()[at] if s["index"] is not None else at
    y = torch.bmm(x[rows.view(-1)].view(len(chosen), s["most"], -1), w if c["transposed"] else w.transpose(1, 2))
    y = _epilogue(s, y[nth, slot - first[nth]], chosen[nth])
    return dict(zip(("codes", "scales"), _quantize(y))) if c["out"] == "fp8" else y.to(DTYPES[c["out"]])


def _placed(s, values, T, k):
    """values [T * k, H] of the choices, at their slots: plain rows or codes and scales."""
    c, out = s["case"], s["out"]
    if s["slots"] is None:
        to = torch.arange(T, device=values.device)
    else:
        flat = s["slots"].view(-1).long()
        to = torch.where(flat >= 0, flat, T * k)         # choices that fell away: one row more, cut off
    if c["out"] != "fp8":
        rows = torch.cat([torch.zeros_like(out), out[:1]])
        rows[to] = values.to(out.dtype)
        return rows[:-1]
    codes, scales = _quantize(values)
    q = torch.zeros(len(out[0]) + 1, codes.shape[1], dtype=torch.uint8, device=codes.device)
    q[to] = codes.view(torch.uint8)
    f = torch.zeros(len(out[0]) + 1, scales.shape[1], device=codes.device)
    f[to] = scales
    return dict(codes=q[:-1].view(torch.float8_e4m3fn), scales=f[:-1])


def _plain_dispatch(s):
    T, k = s["case"]["tokens"], s["case"]["k"]
    x = s["x"].float()
    return _placed(s, x.repeat_interleave(k, 0) if k else x, T, k)


def _taken(s):
    """The choices' rows of y [T, k, H], zeros where a choice fell away."""
    y = s["y"][s["slots"].clamp(min=0).long()].float()
    return torch.where((s["slots"] >= 0)[..., None], y, torch.zeros((), device=y.device))


def _plain_combine(s):
    out = (s["weights"][..., None] * _taken(s)).sum(1)
    if s["x"] is not None:
        out = out + s["x"].float()
    return out.to(s["y"].dtype)


def _plain_combine_grad(s):
    T, k = s["case"]["tokens"], s["case"]["k"]
    g = s["x"].float()
    dy = _placed(s, (s["weights"][..., None] * g[:, None]).view(T * k, -1), T, k)
    return dict(dy=dy, dweights=(g[:, None] * _taken(s)).sum(2))


def _plain_route_grad(s):
    c = s["case"]
    w, dw, ids = s["weights"], s["dweights"], s["ids"].long()
    dot = (w * dw).sum(1, keepdim=True)
    if c["renormalize"]:
        d = torch.zeros(s["logits"].shape, device=w.device)
        own_part = w * (dw - dot)
    else:
        v = s["logits"].float()
        p = torch.exp(v - v.amax(1, keepdim=True))
        d = -torch.nan_to_num(p / p.sum(1, keepdim=True)) * dot
        own_part = w * dw
    # choices that fell away add nothing
    return d.scatter_add(1, ids.clamp(min=0), torch.where(ids >= 0, own_part, torch.zeros_like(own_part))).to(s["logits"].dtype)


# ---- the library's kernels -------------------------------------------------------------------------------------------

def _values(q):
    """A quantised result's codes and scales in the types of the values they stand for."""
    return dict(codes=q.codes.view(torch.float8_e4m3fn), scales=q.scales.view(torch.float32)[:, :_blocks(q.cols)])


def _own(s):
    from lossless_nvfp4_scale_gb300 import ops
    c = s["case"]
    if c["op"] == "route_grad":
        return ops.route_grad(s["logits"], s["ids"], s["weights"], s["dweights"], renormalize=c["renormalize"])
    if c["op"] == "combine":
        return ops.combine(s["y"], s["slots"], s["weights"], residual=s["x"])
    if c["op"] == "matmul":
        depth = c["rows"] if c["transposed"] else c["cols"]
        y = ops.fp8_matmul(ops.Quantized(ops.FP8, s["x"], s["x_scales"], depth), s["w"], s["w_scales"],
                           expert_start=s["start"], rows=s["index"], bias=s["bias"], activation=c["act"], gated=c["gated"],
                           row_scale=s["row_scale"], residual=s["residual"], transposed=c["transposed"],
                           out=ops.FP8 if c["out"] == "fp8" else DTYPES[c["out"]])
        return _values(y) if c["out"] == "fp8" else y
    out = ops.Quantized(ops.FP8, *s["out"], c["cols"]) if c["out"] == "fp8" else s["out"]
    if c["op"] == "combine_grad":
        dy, dweights = ops.combine_grad(s["x"], s["y"], s["slots"], s["weights"], out=out)
        return dict(dy=_values(dy) if c["out"] == "fp8" else dy, dweights=dweights)
    y = ops.dispatch(s["x"], s["slots"], out=out) if c["k"] else ops.quantize(s["x"], ops.FP8, out=out)
    return _values(y) if c["out"] == "fp8" else y


def run(state):
    if own:
        return _own(state)
    return {"matmul": _plain_matmul, "dispatch": _plain_dispatch, "combine": _plain_combine,
            "combine_grad": _plain_combine_grad, "route_grad": _plain_route_grad}[state["case"]["op"]](state)


# ---- work and the definition in 64 bits ------------------------------------------------------------------------------

def _row_bytes(kind, cols):
    return _up(cols, 32) + 4 * _blocks(cols) if kind == "fp8" else cols * SIZES[kind]


def work(case):
    if case["op"] == "route_grad":
        T, E, k = case["tokens"], case["experts"], case["k"]
        return {"bytes": T * E * SIZES[case["dtype"]] * (1 if case["renormalize"] else 2) + 12 * T * k, "flops": 5 * T * E}
    if case["op"] != "matmul":
        T, H, k, row = case["tokens"], case["cols"], case["k"], case["cols"] * SIZES[case["dtype"]]
        if case["op"] == "dispatch":
            n = T * max(k, 1)
            return {"bytes": T * row + n * _row_bytes(case["out"], H) + 4 * T * k, "flops": 3 * T * H}
        if case["op"] == "combine":
            return {"bytes": T * row * (k + (2 if case["residual"] else 1)) + 8 * T * k, "flops": 2 * T * k * H}
        return {"bytes": T * row * (k + 1) + T * k * (_row_bytes(case["out"], H) + 12), "flops": 3 * T * k * H}
    E, S, N, K = case["active"], case["slots"], case["rows"], case["cols"]
    depth, F = (N, K) if case["transposed"] else (K, N // 2 if case["gated"] else N)
    T = max(1, S // 4) if case["gather"] else S
    return {"bytes": E * (N * K + 4 * _blocks(N) * _blocks(K)) + T * _row_bytes("fp8", depth) + S * _row_bytes(case["out"], F)
            + (2 * E * N if case["bias"] else 0) + (S * (2 * F + 4) if case["residual"] else 0) + (4 * S if case["gather"] else 0),
            "flops": 2 * S * N * K}


def _exact_quantize(y):
    """Row by row of blocks: the scale that takes the largest to 448, and the nearest codes."""
    rows, cols = y.shape
    codes, scales = torch.zeros(rows, _up(cols, 32), dtype=torch.float64, device=y.device), []
    for b in range(0, cols, BLOCK):
        part = y[:, b:b + BLOCK]
        scale = torch.maximum(part.abs().max(1, keepdim=True).values / 448, torch.full((), 2.0 ** -126, dtype=torch.float64, device=y.device))
        codes[:, b:b + part.shape[1]] = (part / scale).to(torch.float8_e4m3fn).double()
        scales.append(scale)
    return dict(codes=codes, scales=torch.cat(scales, 1))


def _exact_rows(s, values):
    """What each slot gets: values of (token, choice) pairs [T, k, H], zeros for slots that nobody has."""
    c = s["case"]
    if s["slots"] is None:
        return _exact_quantize(values[:, 0])
    out = torch.zeros(c["tokens"] * c["k"], c["cols"], dtype=torch.float64, device=values.device)
    used = s["slots"] >= 0
    out[s["slots"][used].long()] = values[used]
    if c["out"] != "fp8":
        return out
    q = _exact_quantize(out)
    q["scales"][~torch.isin(torch.arange(len(out), device=out.device), s["slots"])] = 0
    return q


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route_grad":
        # the gradient of sum(dweights * weights(logits)) by its definition: d weight_j / d logit_e
        v, ids = s["logits"].double(), s["ids"].long()
        p = torch.nan_to_num(torch.softmax(v, 1))
        on = ids >= 0
        w = torch.where(on, p.gather(1, ids.clamp(min=0)), torch.zeros_like(p[:, :1]))
        total = w.sum(1, keepdim=True) if case["renormalize"] else torch.ones_like(w[:, :1])
        w = torch.nan_to_num(w / total)
        d = torch.zeros_like(p)
        for j in range(case["k"]):
            dw = s["dweights"][:, j:j + 1].double() * w[:, j:j + 1]
            if case["renormalize"]:
                for i in range(case["k"]):
                    d.scatter_add_(1, ids[:, i:i + 1].clamp(min=0), torch.where(on[:, i:i + 1], -dw * w[:, i:i + 1], torch.zeros_like(dw)))
            else:
                d -= dw * p
            d.scatter_add_(1, ids[:, j:j + 1].clamp(min=0), torch.where(on[:, j:j + 1], dw, torch.zeros_like(dw)))
        return d
    if case["op"] == "dispatch":
        return _exact_rows(s, s["x"].double()[:, None].expand(-1, max(case["k"], 1), -1))
    if case["op"] != "matmul":
        out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device=s["y"].device)
        dw = torch.zeros(case["tokens"], case["k"], dtype=torch.float64, device=s["y"].device)
        for j in range(case["k"]):
            used = s["slots"][:, j] >= 0
            rows = s["y"][s["slots"][used, j].long()].double()
            out[used] += s["weights"][used, j, None].double() * rows
            if case["op"] == "combine_grad":
                dw[used, j] = (rows * s["x"][used].double()).sum(1)
        if case["op"] == "combine":
            return out + s["x"].double() if case["residual"] else out
        return dict(dy=_exact_rows(s, s["weights"].double()[..., None] * s["x"].double()[:, None]), dweights=dw)
    dev = s["x"].device
    S, N, K = case["slots"], case["rows"], case["cols"]
    depth, F = (N, K) if case["transposed"] else (K, N)
    start = s["start"].tolist() if s["start"] is not None else [0, S]
    codes, scales = s["x"].view(torch.float8_e4m3fn)[:, :depth].double(), s["x_scales"].view(torch.float32).double()
    source = s["index"].long() if s["index"] is not None else torch.arange(S, device=dev)
    y = torch.zeros(S, F, dtype=torch.float64, device=dev)
    for i in range(case["experts"]):
        mine = slice(start[i], start[i + 1])
        if start[i] == start[i + 1]:
            continue
        w, sw = s["w"][i].double(), s["w_scales"][i].double()
        if case["transposed"]:
            w, sw = w.T, sw.T
        for b in range(_blocks(depth)):
            part = slice(b * BLOCK, min((b + 1) * BLOCK, depth))
            column = sw[torch.arange(F, device=dev) // BLOCK, b]
            y[mine] += codes[source[mine], part] @ w[:, part].T * scales[source[mine], b, None] * column
        if s["bias"] is not None:
            y[mine] += s["bias"][i].double()
    z = y[:, :F // 2] if case["gated"] else y
    a = {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
         "gelu": lambda: z * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))}[case["act"]]()
    if case["gated"]:
        a = a * y[:, F // 2:]
    if s["residual"] is not None:
        a = a * s["row_scale"].double()[:, None] + s["residual"].double()
    return _exact_quantize(a) if case["out"] == "fp8" else a
