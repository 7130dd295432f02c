"""What the binding of the few-token layer and MoeBuffers.experts take and refuse,
with stand-ins for device tensors and for the library: nothing is launched."""
from __future__ import annotations

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m


class Device:
    """A tensor of n bytes as the binding looks at one."""

    def __init__(self, n, cuda=True):
        self.nbytes, self.is_cuda = n, cuda

    def is_contiguous(self):
        return True

    def is_pinned(self):
        return not self.is_cuda

    def numel(self):
        return self.nbytes

    def element_size(self):
        return 1

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def launched(monkeypatch):
    from combine_expert_count_gb300 import build
    build.build()
    m.sizes_query(m.make_shape(1, 2, 4, 2, 256))
    calls = []

    class Lib:
        @staticmethod
        def moe_layer_few(*a):
            calls.append(a)
            return m.MOE_OK
    monkeypatch.setattr(m, "_lib", Lib)
    monkeypatch.setattr(m, "_raw_stream", lambda stream: 0)
    return calls


@pytest.mark.parametrize("x_cuda", [True, False])
def test_few_takes_pinned_x_but_no_pinned_out(launched, x_cuda):
    """The kernels keep x's coding in out."""
    sh, big = m.make_shape(1, 2, 4, 2, 256), Device(1 << 20)

    def call(out):
        m.moe_layer_few(sh, 128, Device(1 << 20, x_cuda), *[big] * 8, out, big)
    with pytest.raises(ValueError, match="out"):
        call(Device(1 << 20, cuda=False))
    with pytest.raises(ValueError, match="out"):
        call(None)
    assert not launched
    call(big)
    assert len(launched) == 1


@pytest.fixture
def experts(monkeypatch):
    """MoeBuffers of E = 4 experts and hidden 256, and the widths its products get."""
    widths = []
    monkeypatch.setattr(m, "moe_expert_gemm_swiglu", lambda sh, inter, k, *a: widths.append(inter))
    monkeypatch.setattr(m, "moe_expert_gemm", lambda sh, n, k, *a: widths.append(k))
    from combine_expert_count_gb300 import build
    build.build()
    return m.MoeBuffers(1, 2, 4, 2, 256, device="cpu"), widths


@pytest.mark.parametrize("shape,dtype", [
    ((4, 256, 384), torch.uint8), ((4 * 256, 384), torch.uint8), ((4 * 256 * 384,), torch.uint8),
    ((4, 256, 384), torch.float8_e4m3fn), ((4 * 256 * 96,), torch.int32), ((4, 256, 96), torch.int32),
])
def test_the_experts_width_is_that_of_the_bytes_given(experts, shape, dtype):
    buf, widths = experts
    buf.experts(None, None, torch.empty(shape, dtype=dtype), None)
    assert widths == [384, 384]


@pytest.mark.parametrize("n", [0, 4 * 256 * 100, 4 * 256 * 128 + 1])
def test_flat_weights_of_no_whole_width_are_refused(experts, n):
    buf, widths = experts
    with pytest.raises(ValueError, match="w2_q"):
        buf.experts(None, None, torch.empty(n, dtype=torch.uint8), None)
    assert not widths and not buf._h
