"""The rule of the 16-bit products (csrc/linear.h) for a size: which kernel, and in how
many CTAs.  The rule is plain host code; it is compiled here with the C++ compiler."""
from __future__ import annotations

import collections
import ctypes
import functools
import os
import subprocess
import tempfile

from combine_expert_count_gb300 import build

Plan = collections.namedtuple("Plan", "width at parts stages")

_SHIM = """
#include "linear_plan.h"
extern "C" void plan(int64_t rows, int64_t n, int64_t k, int pair, int f32, int sms, int *out) {
    const moe::LinearPlan p = moe::linear_plan(rows, n, k, pair != 0, f32 != 0, sms);
    out[0] = p.width; out[1] = p.at; out[2] = p.parts; out[3] = p.stages;
}
"""


@functools.cache
def _shim() -> ctypes.CDLL:
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(_SHIM)
        subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-shared", "-fPIC",
                        f"-I{build.CSRC}", src, "-o", so], check=True)
        h = ctypes.CDLL(so)
    h.plan.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 3 + [ctypes.c_void_p]
    h.plan.restype = None
    return h


def plan(rows: int, n: int, k: int, pair: bool, f32: bool, sms: int = 152) -> Plan:
    out = (ctypes.c_int * 4)()
    _shim().plan(rows, n, k, pair, f32, sms, out)
    return Plan(*out)


def way(p: Plan) -> str:
    """ "16" .. "128": rows of a CTA; "tiles"; with "/2" .. "/8" where k is shared. """
    return ("tiles" if p.width else str(p.at)) + (f"/{p.parts}" if p.parts > 1 else "")
