"""Buffers of another type than a call's values are refused before anything is launched:
fp16 rows would be read as bf16, and int64 ids written as pairs of int32."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from .test_around_abi import CALLS, NEEDS, Device
from .test_operators_abi import lib  # noqa: F401

TYPES = {"fp32": ("logits", "topk_w", "s"), "int32": ("topk_idx", "status"), "e4m3": ("q",)}
OTHERS = {"bf16": (torch.float16, torch.float32, torch.float64),
          "e4m3": (torch.float16, torch.float32, torch.float64),
          "fp32": (torch.float16, torch.float64),
          "int32": (torch.float16, torch.float32, torch.float64, torch.int64)}
OWN = {"bf16": torch.bfloat16, "fp32": torch.float32, "int32": torch.int32,
       "e4m3": torch.float8_e4m3fn}


def holds(call, name):
    if call == "moe_topk" and name == "bias":
        return "fp32"
    return next((t for t, names in TYPES.items() if name in names), "bf16")


@pytest.fixture
def launched(lib, monkeypatch):  # noqa: F811
    seen = []

    class Lib:
        def __getattr__(self, fn):
            return lambda *a: seen.append(fn) or m.MOE_OK
    monkeypatch.setattr(m, "_lib", Lib())
    monkeypatch.setattr(m, "_stream_on", lambda stream, device: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return seen


@pytest.mark.parametrize("call", list(CALLS))
def test_other_types_are_refused(launched, call):
    sh = m.make_shape(1, 2, 4, 2, 256)
    good = {k: Device(2 * n, dtype=OWN[holds(call, k)]) for k, n in NEEDS[call].items()}
    CALLS[call](sh, good)
    assert launched == [call]
    for name, n in NEEDS[call].items():
        for dtype in OTHERS[holds(call, name)]:
            if call == "moe_linear" and name == "y" and dtype == torch.float32:
                continue  # the fp32 output
            with pytest.raises(ValueError, match=f"^{name}: {dtype}, .*{holds(call, name)}"):
                CALLS[call](sh, {**good, name: Device(2 * n, dtype=dtype)})
    assert launched == [call]


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("raw", [torch.uint8, torch.int16, torch.int32])
def test_raw_views_hold_any(launched, call, raw):
    CALLS[call](m.make_shape(1, 2, 4, 2, 256),
                {k: Device(n, dtype=raw) for k, n in NEEDS[call].items()})
    assert launched == [call]


def test_empty_buffers_are_of_any_type(launched):
    e = Device(0, dtype=torch.float64)
    m.moe_topk(m.make_shape(1, 0, 8, 2, 128), e, e, e)
    assert launched == ["moe_topk"]
