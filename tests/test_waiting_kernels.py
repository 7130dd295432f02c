"""Kernels that are on the GPU before the one before them has ended (they wait for it with
griddepcontrol.wait) read what it may write by plain loads: the read-only path, by name or
through a const pointer that is declared unaliased, is for data that no one writes while
the kernel lives."""
from __future__ import annotations

import glob
import os
import re

import pytest

from combine_expert_count_gb300 import build

SOURCES = {os.path.basename(f): open(f).read()
           for f in glob.glob(os.path.join(build.CSRC, "*.cu*"))}
WAITING = sorted(n for n, s in SOURCES.items() if "griddepcontrol.wait" in s)
# what no kernel of the library writes: the scales of weights
NEVER_WRITTEN = ("ws", "wu")


def read_only(source: str) -> list[str]:
    loads = [re.sub(r"^min\((.*)", r"\1", a) for a in re.findall(r"__ldg\(\s*([^;]*)", source)]
    loads = [a for a in loads if re.match(r"\w+", a).group(0) not in NEVER_WRITTEN]
    return loads + re.findall(r"const \w+ \*\s*__restrict__ \w+", source) + \
        re.findall(r"ld\.global\.nc\S*", source)


def function(source: str, name: str) -> str:
    at = source.index(name)
    return source[at:source.index("\n}\n", at)]


def test_the_waiting_kernels_are_known():
    assert WAITING == ["block.cu", "dispatch.cu", "experts.cu", "linear.cu", "linear_tiles.cuh",
                       "norm.cu", "thin.cu", "topk.cu"]


@pytest.mark.parametrize("name", [n for n in WAITING if n != "dispatch.cu"])
def test_plain_loads(name):
    assert read_only(SOURCES[name]) == []


def test_dispatch_behind_the_routing_kernel():
    """Of its kernels one waits; x, which it reads before, is complete by then."""
    s = SOURCES["dispatch.cu"]
    assert read_only(function(s, "__device__ __forceinline__ void dest_rows(")) == []
    kernel = function(s, "    k_quant_pack_staged(")
    assert read_only(kernel) == ["const uint16_t *__restrict__ x"]
