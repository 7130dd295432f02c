"""The products' own rule (csrc/plan.h) for a size: which kernel, and in how many
CTAs.  The header is plain host code; it is compiled here with the C++ compiler."""
from __future__ import annotations

import collections
import ctypes
import functools
import os
import subprocess
import tempfile

from combine_expert_count_gb300 import build

Plan = collections.namedtuple("Plan", "few units wide tiles parts")

_SHIM = """
#include "plan.h"
extern "C" void plan(int64_t N, int64_t cap, int64_t E, int64_t n, int64_t k, int pair, int sms,
                     int64_t *out) {
    const moe::ProductPlan p = moe::product_plan(N, cap, E, n, k, pair != 0, sms);
    out[0] = p.few; out[1] = p.units; out[2] = p.wide; out[3] = p.tiles; out[4] = p.parts;
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
    h.plan.argtypes = [ctypes.c_int64] * 5 + [ctypes.c_int] * 2 + [ctypes.c_void_p]
    h.plan.restype = None
    return h


def sms() -> int:
    import torch
    return torch.cuda.get_device_properties(0).multi_processor_count


def plan(N: int, cap: int, E: int, n: int, k: int, swiglu: bool, sm_count: int) -> Plan:
    """n counts all outputs, gate and up together."""
    out = (ctypes.c_int64 * 5)()
    _shim().plan(N, cap, E, n, k, swiglu, sm_count, out)
    return Plan(bool(out[0]), *out[1:])


def way(p: Plan) -> str:
    """ "few": the kernels for few rows; "shared": tiles that two CTAs share;
    "tiles": a CTA to a tile. """
    return "few" if p.few else "shared" if p.parts == 2 else "tiles"
