"""CPU checks of the expert-layer operators' C ABI (include/csf_ops.h): the
symbols, the structs that ops.py packs, and the refusals that return before
any CUDA call.  No GPU needed."""
import os
import re
import struct
import subprocess

import pytest

from lossless_nvfp4_scale_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG, SIZE, UNSUPPORTED = 1, 2, 3


@pytest.fixture(scope="module")
def ops():
    build.ensure_built()
    from lossless_nvfp4_scale_gb300 import ops as mod
    return mod


def test_every_declared_symbol_is_exported(ops):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "csf_ops.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(csf_[a-z0-9_]+)\s*\(", text))
    assert names == {"csf_rms_norm", "csf_route", "csf_route_scratch_bytes", "csf_expert_matmul"}
    for n in names:
        assert hasattr(ops.lib, n), n


def test_packed_structs_match_the_header(ops, tmp_path):
    """The byte offset of every field that ops.py packs, against the C compiler's."""
    structs = {"csf_rows": "kind cols rows codes code_stride scales scale_stride tensor_scale".split(),
               "csf_rms_norm_args": "x x_stride residual residual_stride sum_out sum_stride weight dtype eps out".split(),
               "csf_route_args": ("logits logits_stride dtype tokens experts k renormalize ids weights expert_start "
                                  "rows slots scratch scratch_bytes").split(),
               "csf_expert_matmul_args": ("x rows slots experts n w w_scales expert_start expert_start_is_int64 alpha "
                                          "bias bias_dtype act gated row_scale residual residual_stride residual_dtype "
                                          "out_dtype out out_stride out_rows error_word").split()}
    lines = [f'printf("{s} {f} %zu\\n", offsetof({s}, {f}));' for s, fs in structs.items() for f in fs]
    lines += [f'printf("{s} size %zu\\n", sizeof({s}));' for s in structs]
    c = tmp_path / "o.c"
    c.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "csf_ops.h"\nint main(void) {' + "".join(lines) + "}")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(c), "-o",
                    str(tmp_path / "o")], check=True)
    want = {}
    for line in subprocess.run([str(tmp_path / "o")], capture_output=True, text=True, check=True).stdout.splitlines():
        s, f, at = line.split()
        want.setdefault(s, {})[f] = int(at)

    def offsets(fmt):
        at, out = 0, []
        for ch in fmt:
            size = struct.calcsize(ch)
            at = -(-at // size) * size
            out.append(at)
            at += size
        return out

    rows = ops._ROWS
    for s, fmt in (("csf_rows", rows), ("csf_rms_norm_args", ops._RMS_NORM.format[1:]),
                   ("csf_route_args", ops._ROUTE.format[1:]), ("csf_expert_matmul_args", ops._EXPERT_MATMUL.format[1:])):
        flat = [k for f in structs[s] for k in ([f] + [None] * (len(rows) - 1) if f in ("out", "x", "out_rows")
                                                and s in ("csf_rms_norm_args", "csf_expert_matmul_args")
                                                and not (f == "x" and s == "csf_rms_norm_args")
                                                and not (f == "out" and s == "csf_expert_matmul_args") else [f])]
        got = offsets(fmt)
        assert len(flat) == len(got), s
        for f, at in zip(flat, got):
            assert f is None or want[s][f] == at, (s, f)
        assert struct.calcsize("@" + fmt) == want[s]["size"], s


def rows(kind=0, cols=256, n=4, codes=256, cs=None, scales=512, ss=16, ts=0):
    return (kind, cols, n, codes, cs if cs is not None else (cols // 2 if kind == 0 else cols), scales, ss, ts)


def test_rms_norm_refusals(ops):
    def call(x=256, xs=256, res=0, rs=0, out_sum=0, ss=0, w=256, dtype=0, eps=1e-6, out=None):
        return ops.lib.csf_rms_norm(ops._RMS_NORM.pack(x, xs, res, rs, out_sum, ss, w, dtype, eps, *(out or rows())), None)

    assert ops.lib.csf_rms_norm(None, None) == ARG
    assert call(dtype=3) == ARG and call(x=0) == ARG and call(w=0) == ARG
    assert call(xs=255) == ARG                                   # rows overlap
    assert call(res=256, rs=100) == ARG and call(out_sum=256, ss=1) == ARG
    assert call(x=257) == ARG and call(dtype=2, x=258) == ARG    # off the element's alignment
    assert call(out=rows(kind=2)) == ARG and call(out=rows(cols=0)) == ARG
    assert call(out=rows(codes=264)) == ARG and call(out=rows(scales=520)) == ARG
    assert call(out=rows(cs=120)) == ARG and call(out=rows(ss=8)) == ARG
    assert call(out=rows(cols=272, cs=136, ss=32)) == ARG         # 272 columns take 144 code bytes
    assert call(out=rows(n=0)) == 0                              # nothing to do


def test_route_refusals(ops):
    def call(logits=256, ls=8, dtype=2, T=4, E=8, k=2, ids=256, w=256, es=256, r=256, s=256, scratch=0, nbytes=0):
        return ops.lib.csf_route(ops._ROUTE.pack(logits, ls, dtype, T, E, k, 1, ids, w, es, r, s, scratch, nbytes), None)

    assert ops.lib.csf_route(None, None) == ARG
    assert call(dtype=7) == ARG and call(T=-1) == ARG and call(E=0) == ARG
    assert call(k=0) == ARG and call(k=9) == ARG                 # more choices than experts
    assert call(logits=0) == ARG and call(ls=7) == ARG and call(ids=0) == ARG and call(es=0) == ARG
    assert call(logits=258) == ARG                               # float32 off its alignment
    assert call(E=1025, ls=1025) == UNSUPPORTED and call(E=64, ls=64, k=33) == UNSUPPORTED
    assert call(T=1 << 30, k=2) == UNSUPPORTED
    need = ops.lib.csf_route_scratch_bytes(513, 8)
    assert ops.lib.csf_route_scratch_bytes(512, 8) == 0 and need >= 10 * 8 * 4
    assert call(T=513, scratch=0, nbytes=need) == ARG and call(T=513, scratch=256, nbytes=need - 1) == SIZE


def test_expert_matmul_refusals(ops):
    def call(x=None, ri=0, S=4, E=2, N=256, w=256, ws=256, es=256, es64=0, alpha=0, bias=0, bdt=0, act=0, gated=0,
             rscale=0, res=0, rstr=0, rdt=0, odt=0, out=256, ostr=256, orows=None):
        return ops.lib.csf_expert_matmul(ops._EXPERT_MATMUL.pack(
            *(x or rows()), ri, S, E, N, w, ws, es, es64, alpha, bias, bdt, act, gated, rscale, res, rstr, rdt, odt, out,
            ostr, *(orows or (0,) * 8), 0), None)

    assert ops.lib.csf_expert_matmul(None, None) == ARG
    assert call(x=rows(kind=5)) == ARG and call(x=rows(codes=0)) == ARG
    assert call(E=0) == ARG and call(N=0) == ARG and call(S=-1) == ARG
    assert call(E=8193) == UNSUPPORTED
    assert call(act=4) == ARG and call(act=-1) == ARG
    assert call(x=rows(cols=48, cs=32)) == UNSUPPORTED           # K off 32
    assert call(x=rows(kind=1, cols=192, cs=192)) == UNSUPPORTED  # MXFP8: K off 128
    assert call(gated=1, N=384) == UNSUPPORTED                   # halves off 128 rows
    assert call(es=0) == ARG                                     # two experts, no expert_start
    assert call(S=5) == ARG                                      # more slots than x rows, no index
    assert call(w=0) == ARG and call(w=272) == ARG and call(ws=0) == ARG and call(ws=264) == ARG
    assert call(bias=256, bdt=9) == ARG and call(res=256, rstr=255) == ARG and call(res=256, rstr=256, rdt=5) == ARG
    assert call(odt=3) == ARG and call(ostr=255) == ARG
    assert call(out=0) == ARG                                    # neither a plain nor a quantised output
    assert call(out=0, orows=rows(cols=255, n=4)) == ARG and call(out=0, orows=rows(cols=256, n=3)) == ARG
    assert call(S=0) == 0


def test_binding_refusals_without_a_gpu(ops):
    import torch
    x = torch.zeros(4, 256)
    with pytest.raises(ops.CsfError, match="CUDA"):
        ops.rms_norm(x, torch.zeros(256), ops.NVFP4)
    with pytest.raises(ops.CsfError, match="rows"):
        ops.rms_norm(x[0], torch.zeros(256), ops.NVFP4)
    with pytest.raises(ops.CsfError, match="k must be"):
        ops.route(x, 0)
    with pytest.raises(ops.CsfError, match="k must be"):
        ops.route(x, 33)
    with pytest.raises(ops.CsfError, match="NVFP4 or MXFP8"):
        ops.empty_quantized(2, 4, 256, device="cpu")
    q = ops.empty_quantized(ops.NVFP4, 4, 256, device="cpu")
    assert q.codes.shape == (4, 128) and q.scales.shape == (4, 16)
    with pytest.raises(ops.CsfError, match="CUDA"):
        ops.expert_matmul(q, torch.zeros(1, 8, 128, dtype=torch.uint8), torch.zeros(1))


def test_pointers_off_their_elements_are_refused(ops):
    """Every pointer that a kernel reads or writes by elements, one byte or one half element off."""
    def norm(**kw):
        a = dict(x=256, xs=256, res=0, rs=0, out_sum=0, ss=0, w=256, dtype=0, eps=1e-6, ts=0)
        a.update(kw)
        return ops.lib.csf_rms_norm(ops._RMS_NORM.pack(*list(a.values())[:9], *rows(ts=a["ts"])), None)

    assert norm(ts=258) == ARG and norm(res=257, rs=256) == ARG and norm(out_sum=257, ss=256) == ARG

    def route(**kw):
        a = dict(logits=256, ls=8, dtype=2, T=4, E=8, k=2, renormalize=1, ids=256, w=256, es=256, r=256, s=256, scratch=0, n=0)
        a.update(kw)
        return ops.lib.csf_route(ops._ROUTE.pack(*a.values()), None)

    for name in ("ids", "w", "es", "r", "s"):
        assert route(**{name: 258}) == ARG, name

    def product(**kw):
        a = dict(ri=0, S=4, E=2, N=256, w=256, ws=256, es=256, es64=0, alpha=0, bias=0, bdt=0, act=0, gated=0, rscale=0,
                 res=0, rstr=256, rdt=0, odt=0, out=256, ostr=256)
        err, orows = kw.pop("err", 0), kw.pop("orows", (0,) * 8)
        a.update(kw)
        return ops.lib.csf_expert_matmul(ops._EXPERT_MATMUL.pack(*rows(), *a.values(), *orows, err), None)

    for name in ("ri", "es", "alpha", "rscale", "err"):
        assert product(**{name: 258}) == ARG, name
    assert product(es=260, es64=1) == ARG
    for dtype, off in ((0, 257), (1, 257), (2, 258)):
        assert product(bias=off, bdt=dtype) == ARG
        assert product(res=off, rdt=dtype) == ARG
        assert product(out=off, odt=dtype) == ARG
    assert product(out=0, orows=rows(ts=258)) == ARG


def test_widths_next_to_32_bits_are_refused(ops):
    """Columns and rows of whole tiles are counted in 32 bits."""
    def product(x, N):
        return ops.lib.csf_expert_matmul(ops._EXPERT_MATMUL.pack(
            *x, 0, 4, 1, N, 256, 256, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 256, 1 << 31, *(0,) * 8, 0), None)

    assert product(rows(), 2 ** 31 - 1) == UNSUPPORTED
    k = 2 ** 31 - 128
    assert product(rows(cols=k, cs=k // 2, ss=k // 16 + 8), 128) == UNSUPPORTED       # strides are multiples of 16


class On:
    """A tensor that says it lies on a CUDA device."""
    def __init__(self, t, device):
        import torch
        self.t, self.device = t, torch.device("cuda", device)

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.device.index

    is_cuda = True


def test_tensors_of_another_device_are_refused(ops):
    import types
    import torch
    x, w = torch.zeros(4, 64), torch.zeros(64)
    with pytest.raises(ops.CsfError, match="residual.*on cuda:0"):
        ops.rms_norm(On(x, 0), On(w, 0), ops.NVFP4, residual=On(x, 1))
    with pytest.raises(ops.CsfError, match="weight.*on cuda:1"):
        ops.rms_norm(On(x, 1), On(w, 0), ops.NVFP4)
    with pytest.raises(ops.CsfError, match="out.*on cuda:0"):
        ops.rms_norm(On(x, 0), On(w, 0), ops.NVFP4, out=ops.empty_quantized(ops.NVFP4, 4, 64, device="cpu"))

    def product(at, **kw):
        codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 16, dtype=torch.uint8)
        weights, sf = torch.zeros(2, 8, 32, dtype=torch.uint8), torch.zeros(2 * 512, dtype=torch.uint8)
        start = torch.zeros(3, dtype=torch.int32)
        q = ops.Quantized(ops.NVFP4, On(codes, 0), On(scales, at.get("scales", 0)), 64)
        ops.expert_matmul(q, On(weights, at.get("w", 0)), On(sf, at.get("sf", 0)), On(start, at.get("start", 0)), **kw)

    for at, match in ((dict(scales=1), "x: codes and scales"), (dict(w=1), "w must"), (dict(sf=1), "w_scales"), (dict(start=1), "expert_start")):
        with pytest.raises(ops.CsfError, match=match + ".*on cuda:0"):
            product(at)
    for name, t in (("rows", torch.zeros(4, dtype=torch.int32)), ("residual", torch.zeros(4, 8)), ("out", torch.zeros(4, 8)),
                    ("alpha", torch.zeros(2)), ("bias", torch.zeros(2, 8)), ("row_scale", torch.zeros(4))):
        with pytest.raises(ops.CsfError, match=name + ".*on cuda:0"):
            product({}, **{"out": On(torch.zeros(4, 8), 0), name: On(t, 1)})
    with pytest.raises(ops.CsfError, match="the stream is on cuda:1, the tensors on cuda:0"):
        ops.route(On(x, 0), 2, stream=types.SimpleNamespace(device=torch.device("cuda", 1)))


def test_a_call_runs_on_its_tensors_device(ops, monkeypatch):
    """The device is made current around the library call where it is not; the stream is that device's."""
    import contextlib
    import torch
    current, log = [0], []

    @contextlib.contextmanager
    def device(i):
        was, current[0] = current[0], i
        yield
        current[0] = was

    monkeypatch.setattr(ops, "_current_device", lambda: current[0])
    monkeypatch.setattr(ops, "_raw_stream", lambda i: 100 + i)
    monkeypatch.setattr(torch.cuda, "device", device)
    for d in (0, 1):
        ops._launch(lambda args, stream: log.append((args, stream, current[0])) or 0, b"x", d, "call")
    assert log == [(b"x", 100, 0), (b"x", 101, 1)] and current == [0]
    with pytest.raises(ops.CsfError, match="call"):
        ops._launch(lambda args, stream: ARG, b"", 1, "call")
    assert current == [0]
