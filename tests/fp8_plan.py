"""The library's own choice of a kernel for a product of FP8 rows (csrc/csf_fp8_plan.h), compiled for the host."""
import ctypes
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ONE, TWO, ONE_SHARED, TWO_SHARED = range(4)

SOURCE = r"""
#include "csf_fp8_plan.h"
extern "C" void plan(int sms, long long slots, int experts, int F, int blocks, int gated, long long *out) {
    const csfk::f8::Plan p = csfk::f8::plan_of({sms, slots, experts, F, blocks, gated != 0});
    out[0] = p.shape, out[1] = p.split, out[2] = p.stages, out[3] = p.smem, out[4] = p.most_tiles, out[5] = p.nt, out[6] = p.tile_step;
}
"""
_lib = None


class Plan:
    def __init__(self, sms, slots, experts, F, depth, gated=False):
        global _lib
        if _lib is None:
            with tempfile.TemporaryDirectory() as d:
                src, so = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
                with open(src, "w") as f:
                    f.write(SOURCE)
                subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-Wall", "-Werror",
                                "-I" + os.path.join(ROOT, "lossless_nvfp4_scale_gb300", "csrc"), src, "-o", so], check=True)
                _lib = ctypes.CDLL(so)
        out = (ctypes.c_longlong * 7)()
        _lib.plan(sms, ctypes.c_longlong(slots), experts, F, -(-depth // 128), gated, out)
        self.shape, self.split, self.stages, self.smem, self.most_tiles, self.nt, self.tile_step = out
