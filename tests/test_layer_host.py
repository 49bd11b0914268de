"""CPU checks of csf_layer.h's C ABI: the symbols, the structs that ops.py
packs, and the refusals that return before any CUDA call.  No GPU needed."""
import os
import re
import struct
import subprocess

import pytest

from lossless_nvfp4_scale_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG, UNSUPPORTED = 1, 3
FP8 = 3


@pytest.fixture(scope="module")
def ops():
    build.ensure_built()
    from lossless_nvfp4_scale_gb300 import ops as mod
    return mod


def test_every_declared_symbol_is_exported(ops):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "csf_layer.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(csf_[a-z0-9_]+)\s*\(", text))
    assert names == {"csf_fp8_matmul", "csf_dispatch", "csf_combine", "csf_combine_grad", "csf_route_grad"}
    for n in names:
        assert hasattr(ops.lib, n), n


STRUCTS = {
    "csf_fp8_matmul_args": ("_FP8_MATMUL", "x* rows slots experts n k transposed w w_scales expert_start expert_start_is_int64 bias_dtype bias act "
                                           "gated row_scale residual residual_stride residual_dtype out_dtype out out_stride out_rows* error_word"),
    "csf_dispatch_args": ("_DISPATCH", "x x_stride dtype tokens cols k slots out_count out out_stride out_dtype out_rows* error_word"),
    "csf_combine_args": ("_COMBINE", "y y_stride y_rows y_dtype tokens cols k slots weights residual residual_stride residual_dtype out_dtype out "
                                     "out_stride error_word"),
    "csf_combine_grad_args": ("_COMBINE_GRAD", "g g_stride y y_stride slot_rows g_dtype y_dtype tokens cols k dy_dtype slots weights dy dy_stride "
                                               "dy_rows* dweights error_word"),
    "csf_route_grad_args": ("_ROUTE_GRAD", "logits logits_stride dlogits dlogits_stride dtype tokens experts k ids weights dweights renormalize"),
}


def test_packed_structs_match_the_header(ops, tmp_path):
    """The byte offset and size of every field that ops.py packs, against the C compiler's."""
    lines = []
    for s, (_, fields) in STRUCTS.items():
        for f in fields.replace("*", "").split():
            lines.append(f'printf("{s} {f} %zu %zu\\n", offsetof({s}, {f}), sizeof((({s} *)0)->{f}));')
        lines.append(f'printf("{s} = %zu 0\\n", sizeof({s}));')
    c = tmp_path / "o.c"
    c.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "csf_layer.h"\nint main(void) {' + "".join(lines) + "}")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(c), "-o", str(tmp_path / "o")], check=True)
    want = {}
    for line in subprocess.run([str(tmp_path / "o")], capture_output=True, text=True, check=True).stdout.splitlines():
        s, f, at, size = line.split()
        want[s, f] = int(at), int(size)
    for s, (name, fields) in STRUCTS.items():
        fmt = getattr(ops, name).format[1:]
        at, got = 0, []                              # (offset, size) of each packed item
        for n, ch in re.findall(r"(\d*)(\w)", fmt):
            if ch == "x":
                at += int(n)
                continue
            size = struct.calcsize(ch)
            at = -(-at // size) * size
            got.append((at, size))
            at += size
        items = iter(got)
        for f in fields.split():
            first = next(items)
            if f.endswith("*"):                      # a csf_rows, its items one by one
                for _ in range(len(ops._ROWS) - 1):
                    next(items)
                assert want[s, f[:-1]][0] == first[0], (s, f)
            else:
                assert want[s, f] == first, (s, f)
        assert next(items, None) is None, s
        assert struct.calcsize("@" + fmt) == want[s, "="][0], s


def rows(kind=FP8, cols=256, n=4, codes=256, cs=None, scales=512, ss=16, ts=0):
    return (kind, cols, n, codes, cs if cs is not None else (cols // 2 if kind == 0 else cols), scales, ss, ts)


def test_fp8_matmul_refusals(ops):
    def call(x=None, ri=0, S=4, E=2, n=256, k=256, tr=0, w=256, ws=256, es=256, es64=0, bdt=0, bias=0, act=0, gated=0, rscale=0, res=0, rstr=0,
             rdt=0, odt=0, out=256, ostr=256, orows=None, word=0):
        return ops.lib.csf_fp8_matmul(ops._FP8_MATMUL.pack(*(x or rows()), ri, S, E, n, k, tr, w, ws, es, es64, bdt, bias, act, gated, rscale, res,
                                                           rstr, rdt, odt, out, ostr, *(orows or (0,) * 8), word), None)

    assert ops.lib.csf_fp8_matmul(None, None) == ARG
    for kind in (0, 1, 2, 4):
        assert call(x=rows(kind=kind)) == ARG
    assert call(x=rows(codes=0)) == ARG and call(x=rows(codes=264)) == ARG and call(x=rows(scales=520)) == ARG
    assert call(x=rows(ss=0)) == ARG and call(x=rows(cols=640, ss=16)) == ARG          # five scales take 32 bytes
    assert call(E=0) == ARG and call(n=0) == ARG and call(S=-1) == ARG and call(k=512) == ARG
    assert call(tr=1, n=512) == ARG                              # x has k columns, not n
    assert call(E=8193) == UNSUPPORTED and call(S=1 << 31) == UNSUPPORTED
    assert call(act=4) == ARG and call(act=-1) == ARG
    assert call(x=rows(cols=264, cs=288), k=264) == UNSUPPORTED  # k off 16
    assert call(x=rows(cols=200, cs=224), n=200, tr=1) == UNSUPPORTED
    assert call(gated=1, n=384) == UNSUPPORTED and call(gated=1, tr=1) == UNSUPPORTED
    assert call(es=0) == ARG and call(es=258) == ARG and call(es=260, es64=1) == ARG
    assert call(S=5) == ARG                                      # more slots than x rows, no index
    assert call(ri=258) == ARG and call(w=0) == ARG and call(w=264) == ARG and call(ws=0) == ARG and call(ws=258) == ARG
    assert call(bias=256, bdt=9) == ARG and call(bias=257) == ARG and call(res=256, rstr=255) == ARG and call(res=256, rstr=256, rdt=5) == ARG
    assert call(rscale=258) == ARG and call(word=258) == ARG
    assert call(odt=3) == ARG and call(ostr=255) == ARG and call(out=257) == ARG and call(odt=2, out=258) == ARG
    assert call(out=0) == ARG                                    # neither a plain nor a quantised output
    assert call(out=0, orows=rows(cols=255)) == ARG and call(out=0, orows=rows(n=3)) == ARG and call(out=0, orows=rows(kind=1)) == ARG
    assert call(S=0) == 0


def test_dispatch_refusals(ops):
    def call(x=256, xs=256, dt=0, T=4, H=256, k=2, slots=256, count=8, out=256, ostr=256, odt=0, orows=None, word=0):
        return ops.lib.csf_dispatch(ops._DISPATCH.pack(x, xs, dt, T, H, k, slots, count, out, ostr, odt, *(orows or (0,) * 8), word), None)

    assert ops.lib.csf_dispatch(None, None) == ARG
    assert call(x=0) == ARG and call(x=257) == ARG and call(xs=255) == ARG and call(dt=3) == ARG and call(T=-1) == ARG and call(H=0) == ARG
    assert call(k=0) == ARG and call(slots=258) == ARG and call(count=-1) == ARG and call(slots=0, count=8) == ARG
    assert call(k=1025) == UNSUPPORTED and call(H=(1 << 24) + 1, xs=1 << 25) == UNSUPPORTED
    assert call(ostr=255) == ARG and call(odt=4) == ARG and call(odt=2, out=258) == ARG and call(word=2) == ARG
    assert call(out=0) == ARG and call(out=0, orows=rows(n=7)) == ARG and call(out=0, orows=rows(n=8, cols=255)) == ARG
    assert call(out=0, orows=rows(n=8, kind=2)) == ARG and call(out=0, orows=rows(n=8, ts=2)) == ARG
    assert call(T=0) == 0 and call(T=0, slots=0, count=0) == 0


def test_combine_refusals(ops):
    def call(y=256, ys=256, yr=8, yd=0, T=4, H=256, k=2, slots=256, w=0, res=0, rs=0, rd=0, od=0, out=256, ostr=256, word=0):
        return ops.lib.csf_combine(ops._COMBINE.pack(y, ys, yr, yd, T, H, k, slots, w, res, rs, rd, od, out, ostr, word), None)

    assert ops.lib.csf_combine(None, None) == ARG
    assert call(y=0) == ARG and call(ys=255) == ARG and call(yr=-1) == ARG and call(yd=3) == ARG and call(T=-1) == ARG and call(H=0) == ARG
    assert call(k=0) == ARG and call(slots=0) == ARG and call(slots=258) == ARG and call(w=258) == ARG and call(word=1) == ARG
    assert call(k=1025) == UNSUPPORTED and call(H=(1 << 24) + 1, ys=1 << 25, ostr=1 << 25) == UNSUPPORTED
    assert call(res=256, rs=255) == ARG and call(res=257, rs=256) == ARG and call(res=256, rs=256, rd=7) == ARG
    assert call(out=0) == ARG and call(out=257) == ARG and call(ostr=255) == ARG and call(od=-1) == ARG
    assert call(T=0) == 0


def test_combine_grad_refusals(ops):
    def call(g=256, gs=256, y=256, ys=256, S=8, gd=0, yd=0, T=4, H=256, k=2, dd=0, slots=256, w=0, dy=256, ds=256, drows=None, dw=256, word=0):
        return ops.lib.csf_combine_grad(ops._COMBINE_GRAD.pack(g, gs, y, ys, S, gd, yd, T, H, k, dd, slots, w, dy, ds, *(drows or (0,) * 8), dw, word), None)

    assert ops.lib.csf_combine_grad(None, None) == ARG
    assert call(g=0) == ARG and call(gs=255) == ARG and call(gd=3) == ARG and call(T=-1) == ARG and call(H=0) == ARG and call(S=-1) == ARG
    assert call(y=0) == ARG and call(ys=255) == ARG and call(yd=4) == ARG and call(dw=258) == ARG
    assert call(k=0) == ARG and call(k=1025) == UNSUPPORTED and call(slots=0) == ARG and call(w=258) == ARG and call(word=1) == ARG
    assert call(dy=257) == ARG and call(ds=255) == ARG and call(dd=9) == ARG
    assert call(dy=0, drows=rows(n=7)) == ARG and call(dy=0, drows=rows(n=8, kind=2)) == ARG and call(dy=0, drows=rows(n=8, ts=2)) == ARG
    assert call(T=0) == 0 and call(dy=0, dw=0, y=0) == 0         # nothing is wanted


def test_route_grad_refusals(ops):
    def call(lg=256, ls=8, out=256, os_=8, dt=2, T=4, E=8, k=2, ids=256, w=256, dw=256, re_=0):
        return ops.lib.csf_route_grad(ops._ROUTE_GRAD.pack(lg, ls, out, os_, dt, T, E, k, ids, w, dw, re_), None)

    assert ops.lib.csf_route_grad(None, None) == ARG
    assert call(dt=7) == ARG and call(T=-1) == ARG and call(E=0) == ARG and call(k=0) == ARG and call(k=9) == ARG
    assert call(lg=0) == ARG and call(ls=7) == ARG and call(lg=258) == ARG and call(out=0) == ARG and call(os_=7) == ARG and call(out=258) == ARG
    assert call(ids=0) == ARG and call(w=0) == ARG and call(dw=0) == ARG and call(ids=258) == ARG
    assert call(E=1025, ls=1025, os_=1025) == UNSUPPORTED and call(E=64, ls=64, os_=64, k=33) == UNSUPPORTED
    assert call(T=0) == 0


def test_binding_refusals_without_a_gpu(ops):
    import torch
    x, slots, w = torch.zeros(4, 256), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for call in (lambda: ops.quantize(x, ops.FP8), lambda: ops.dispatch(x, slots), lambda: ops.combine(x, slots), lambda: ops.combine_grad(x, x, slots),
                 lambda: ops.route_grad(x, slots, w, w)):
        with pytest.raises(ops.CsfError, match="CUDA"):
            call()
    with pytest.raises(ops.CsfError, match="rows"):
        ops.dispatch(x[0], slots)
    with pytest.raises(ops.CsfError, match="NVFP4"):
        ops.quantize(x, 2)
    with pytest.raises(ops.CsfError, match="CUDA"):
        q = ops.empty_quantized(ops.FP8, 4, 256, device="cpu")
        ops.fp8_matmul(q, torch.zeros(1, 128, 256, dtype=torch.uint8), torch.zeros(1, 1, 2))
    assert q.codes.shape == (4, 256) and q.scales.shape == (4, 16)
    assert ops.empty_quantized(ops.FP8, 3, 641, device="cpu").scales.shape == (3, 32)
    with pytest.raises(ops.CsfError, match="NVFP4 or MXFP8"):    # the FP4 experts' product takes its own kinds
        ops.expert_matmul(q, torch.zeros(1, 128, 128, dtype=torch.uint8), torch.zeros(1 << 16, dtype=torch.uint8))
