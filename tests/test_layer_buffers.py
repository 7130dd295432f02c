"""The buffers that MoeBuffers.experts makes by itself, with the products
replaced by recorders: no GPU."""
from __future__ import annotations

import contextlib
import gc
import weakref

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

N, T, E, R, H = 2, 3, 4, 2, 256


@pytest.fixture(scope="module", autouse=True)
def lib():
    from combine_expert_count_gb300 import build
    build.build()
    return m.lib()


@pytest.fixture
def calls(monkeypatch):
    """(h_q, h_s) of each gate/up product that experts() makes, as weak references."""
    seen = []

    def swiglu(shape, inter, k, a_q, a_s, grp_off, w13_q, w13_s, h_q, h_s, *_):
        seen.append((weakref.ref(h_q), weakref.ref(h_s)))
    monkeypatch.setattr(m, "moe_expert_gemm_swiglu", swiglu)
    monkeypatch.setattr(m, "moe_expert_gemm", lambda *a: None)
    return seen


def weights(inter):
    return (torch.zeros((E, 2 * inter, H), dtype=torch.uint8),
            torch.zeros((E, 2 * inter // 128, H // 128)),
            torch.zeros((E, H, inter), dtype=torch.uint8),
            torch.zeros((E, H // 128, inter // 128)))


def test_a_call_with_another_width_keeps_the_first_ones_buffers(calls):
    """A graph or a stream may still hold them."""
    buf = m.MoeBuffers(N, T, E, R, H, device="cpu")
    for inter in (256, 128, 256):
        buf.experts(*weights(inter))
        gc.collect()
    assert all(ref() is not None for pair in calls for ref in pair)
    for a, b in zip(calls[0], calls[2]):
        assert a() is b()
    for (q, s), inter in zip(calls, (256, 128, 256)):
        assert q().shape == (N, buf.cap, inter) and q().dtype == torch.uint8
        assert s().shape == (N, buf.cap, inter // 128) and s().dtype == torch.float32


@pytest.fixture
def allocated(monkeypatch):
    """The stream that each torch.empty is called on."""
    current, at = [None], []

    @contextlib.contextmanager
    def stream(s):
        before, current[0] = current[0], s if s is not None else current[0]
        yield
        current[0] = before
    empty = torch.empty

    def noted(*a, **k):
        at.append(current[0])
        return empty(*a, **k)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "empty", noted)
    return at


def test_buffers_are_allocated_on_the_calls_stream(calls, allocated):
    buf = m.MoeBuffers(N, T, E, R, H, device="cpu")
    del allocated[:]
    buf.experts(*weights(128), stream="side")
    assert allocated == ["side", "side"]
    buf.experts(*weights(128), stream="side")
    buf.experts(*weights(256))
    assert allocated == ["side", "side", None, None]


def test_partial_rows_are_allocated_on_the_calls_stream(allocated, monkeypatch):
    monkeypatch.setattr(m, "moe_combine_partial_send", lambda *a: None)
    monkeypatch.setattr(m, "moe_combine_partial_recv", lambda *a: None)
    buf = m.MoeBuffers(N, T, E, R, H, device="cpu")
    del allocated[:]
    for _ in range(2):
        buf.combine(None, None, stream="side", calls="partial_separate")
    assert allocated == ["side"]


def test_device_bytes_count_every_width_once(calls):
    buf = m.MoeBuffers(N, T, E, R, H, device="cpu")
    before, rows = buf.device_bytes(), N * buf.cap
    for inter in (128, 256, 128):
        buf.experts(*weights(inter))
    assert buf.device_bytes() == before + rows * (128 + 256) + rows * (1 + 2) * 4
