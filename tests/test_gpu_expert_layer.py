"""The example layer (examples/expert_layer.py): norm, router, routed scale
decode and the experts' products together, against the same layer in 64 bits
on the quantised values that the operators hand on."""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lossless_nvfp4_scale_gb300 import build
    build.ensure_built()
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = mod
    spec.loader.exec_module(mod)
    return mod


def values(codes, scales):
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    v = torch.stack([t[(codes & 15).long()], t[(codes >> 4).long()]], -1).flatten(-2)
    return (v.view(*v.shape[:-1], -1, 16) * scales.view(torch.float8_e4m3fn).double()[..., None]).view(v.shape)


@pytest.mark.parametrize("tokens,k", [(1, 4), (33, 8), (200, 2)])
def test_layer(example, tokens, k):
    csf, ops = example.csf, example.ops
    E, H, I = 16, 320, 256
    layer = example.random_layer(E, H, I, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, H, device="cuda", generator=g).to(torch.bfloat16)
    residual = torch.randn(tokens, H, device="cuda", generator=g).to(torch.bfloat16)
    for w in layer.workspace:
        w.fill_(0x7F)                                    # NaN scales: an expert that was not decoded would show
    y, total = layer(x, residual, k)
    assert torch.isfinite(y).all()

    q, total2 = ops.rms_norm(x, layer.norm_weight, ops.NVFP4, residual=residual, tensor_scale=layer.x_scale)
    assert torch.equal(total, total2)
    h = (x.double() + residual.double())
    assert ((total.double() - h).abs() <= 2.0 ** -8 * h.abs()).all()
    r = ops.route(total @ layer.router.T, k)
    gate_up = values(layer.gate_up, csf.decode(layer.gate_up_scales))
    down = values(layer.down, csf.decode(layer.down_scales))
    xv = values(q.codes, q.scales[:, :H // 16])
    act = ops.expert_matmul(q, layer.gate_up, layer.workspace[0], expert_start=r.expert_start, rows=r.rows,
                            alpha=layer.alpha[0], activation="silu", gated=True, out=ops.NVFP4,
                            out_tensor_scale=layer.act_scale)
    av = values(act.codes, act.scales[:, :I // 16])
    want = torch.zeros(tokens, H, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)                        # the magnitudes that were added up
    exact = torch.zeros(tokens, k, I, dtype=torch.float64, device="cuda")
    for t in range(tokens):
        for j in range(k):
            e, s = int(r.ids[t, j]), int(r.slots[t, j])
            p = (gate_up[e] @ xv[t]) * layer.alpha[0, e].double()
            exact[t, j] = p[:I] * torch.sigmoid(p[:I]) * p[I:]
            scale = layer.alpha[1, e].double() * r.weights[t, j].double()
            want[t] += (down[e] @ av[s]) * scale
            size[t] += (down[e].abs() @ av[s].abs()) * scale.abs()
    # 32-bit sums of 256 terms, bfloat16 output
    assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * size).all()
    # The activation as handed on: half the widest gap between codes is a sixth
    # of a block's largest value, the scale's rounding a sixteenth; a value
    # past 6 * 448 tensor scales, the most that codes and scale can hold, is cut.
    most = 6 * 448 * layer.act_scale.double()
    got = (av * layer.act_scale.double())[r.slots.long()].view(tokens, k, -1, 16)
    exact = exact.view(tokens, k, -1, 16).clamp(-most, most)
    assert ((got - exact).abs() <= exact.abs().amax(-1, keepdim=True) * (1 / 6 + 1 / 16) + 6 * 2.0 ** -10 * 0.005).all()


@pytest.mark.parametrize("tokens,k", [(1, 4), (33, 8), (200, 2)])
def test_layer_with_experts_switched_off(example, tokens, k):
    """Masked routing: tokens with all experts, fewer than k or none.  A token with none gets 0; what is left of the
    others is what the router's choices and the slots' outputs add up to in 64 bits."""
    csf, ops = example.csf, example.ops
    E, H, I = 16, 320, 256
    layer = example.random_layer(E, H, I, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens + 1)
    x = torch.randn(tokens, H, device="cuda", generator=g).to(torch.bfloat16)
    residual = torch.randn(tokens, H, device="cuda", generator=g).to(torch.bfloat16)
    off = torch.rand(tokens, E, device="cuda", generator=g) < 0.5
    off[::3, 1:] = True                                  # one expert left, fewer than k
    off[::4] = True                                      # none
    off[2::5] = False
    junk = [torch.full((tokens * k, H), float("nan"), device="cuda") for _ in range(4)]      # what unwritten rows may hold
    del junk
    y, total = layer(x, residual, k, off=off)
    none = off.all(1)
    assert torch.isfinite(y).all() and (y[none] == 0).all()

    q, _ = ops.rms_norm(x, layer.norm_weight, ops.NVFP4, residual=residual, tensor_scale=layer.x_scale)
    r = ops.route((total @ layer.router.T).masked_fill(off, -float("inf")), k)
    assert ((r.slots >= 0).sum(1) == (~off).sum(1).clamp(max=k)).all()
    act = ops.expert_matmul(q, layer.gate_up, layer.workspace[0], expert_start=r.expert_start, rows=r.rows,
                            alpha=layer.alpha[0], activation="silu", gated=True, out=ops.NVFP4,
                            out_tensor_scale=layer.act_scale)
    down = values(layer.down, csf.decode(layer.down_scales))
    av = values(act.codes, act.scales[:, :I // 16])
    want = torch.zeros(tokens, H, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    for t in range(tokens):
        for j in range(k):
            e, s = int(r.ids[t, j]), int(r.slots[t, j])
            if s < 0:
                continue
            scale = layer.alpha[1, e].double() * r.weights[t, j].double()
            want[t] += (down[e] @ av[s]) * scale
            size[t] += (down[e].abs() @ av[s].abs()) * scale.abs()
    # as above: 32-bit sums of 256 terms, bfloat16 output
    assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * size).all()
