"""Refusals of the products of 16-bit weights, the router's choice and the block's
end: on the host, before anything touches CUDA."""
from __future__ import annotations

import ctypes

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

from .test_operators_abi import BAD, GOOD, each_pointer, lib  # noqa: F401


def test_linear_refusals(lib):
    sh, f = ctypes.byref(m.moe_shape(2, 4, 8, 2, 256, 0)), lib.moe_linear
    # x w bias res y_bf16 y_f32 status: one of the two outputs
    for outs in ((GOOD, None), (None, GOOD)):
        for i in range(7):
            args = [GOOD, GOOD, GOOD, GOOD, *outs, GOOD]
            if args[i] is None:
                continue
            args[i] = BAD
            assert f(sh, 64, 64, 0, *args, None) == m.MOE_EINVAL, i
            args[i] = None
            if i in (0, 1, 4, 5):
                assert f(sh, 64, 64, 0, *args, None) == m.MOE_EINVAL, i
    assert f(sh, 64, 64, 0, *[GOOD] * 7, None) == m.MOE_EINVAL  # both outputs
    ok = [GOOD, GOOD, None, None, GOOD, None, None]
    for n, k, act, code in ((0, 64, 0, m.MOE_EINVAL), (-1, 64, 0, m.MOE_EINVAL),
                            (64, 0, 0, m.MOE_EINVAL), (64, -8, 0, m.MOE_EINVAL),
                            (64, 68, 0, m.MOE_EINVAL), (64, 64, -1, m.MOE_EINVAL),
                            (64, 64, 6, m.MOE_EINVAL), (64, 65544, 0, m.MOE_ENOTSUP),
                            ((1 << 20) + 1, 64, 0, m.MOE_ENOTSUP)):
        assert f(sh, n, k, act, *ok, None) == code, (n, k, act)
    assert f(None, 64, 64, 0, *ok, None) == m.MOE_EINVAL
    assert f(ctypes.byref(m.moe_shape(3, 4, 8, 2, 256, 0)), 64, 64, 0, *ok, None) == m.MOE_EINVAL
    none = ctypes.byref(m.moe_shape(2, 0, 8, 2, 256, 0))
    assert f(none, 64, 64, 0, None, GOOD, None, None, None, None, None, None) == m.MOE_OK


def test_glu_refusals(lib):
    sh, f = ctypes.byref(m.moe_shape(2, 4, 8, 2, 256, 0)), lib.moe_linear_glu
    each_pointer(f, (sh, 64, 64, 2), 5, optional=(2, 4))  # x w13 bias13 h status
    ok = [GOOD, GOOD, None, GOOD, None]
    for n, k, act, code in ((0, 64, 2, m.MOE_EINVAL), (64, 4, 2, m.MOE_EINVAL),
                            (64, 64, 9, m.MOE_EINVAL), ((1 << 19) + 1, 64, 2, m.MOE_ENOTSUP),
                            (1 << 30, 64, 2, m.MOE_ENOTSUP), (64, 1 << 20, 2, m.MOE_ENOTSUP)):
        assert f(sh, n, k, act, *ok, None) == code, (n, k, act)


def test_topk_refusals(lib):
    sh, f = ctypes.byref(m.moe_shape(2, 4, 64, 4, 256, 0)), lib.moe_topk
    each_pointer(f, (sh, 0, 1, 1, 1, 1, 1.0), 4, optional=(1,))  # logits bias idx w
    for score, groups, kept, best, scale, code in (
            (2, 1, 1, 1, 1.0, m.MOE_EINVAL), (-1, 1, 1, 1, 1.0, m.MOE_EINVAL),
            (0, 0, 1, 1, 1.0, m.MOE_EINVAL), (0, 3, 1, 1, 1.0, m.MOE_EINVAL),
            (0, 8, 0, 1, 1.0, m.MOE_EINVAL), (0, 8, 9, 1, 1.0, m.MOE_EINVAL),
            (0, 8, 4, 0, 1.0, m.MOE_EINVAL), (0, 8, 4, 3, 1.0, m.MOE_EINVAL),
            (0, 32, 1, 1, 1.0, m.MOE_EINVAL),                     # two experts for four places
            (0, 64, 4, 2, 1.0, m.MOE_EINVAL), (0, 64, 4, 1, 1.0, m.MOE_ENOTSUP),
            (0, 1, 1, 1, float("nan"), m.MOE_EINVAL), (0, 1, 1, 1, float("inf"), m.MOE_EINVAL)):
        assert f(sh, score, groups, kept, best, 1, scale, *[GOOD] * 4, None) == code, (groups, kept)
    assert f(None, 0, 1, 1, 1, 1, 1.0, *[GOOD] * 4, None) == m.MOE_EINVAL
    none = ctypes.byref(m.moe_shape(2, 0, 64, 4, 256, 0))
    assert f(none, 0, 1, 1, 1, 1, 1.0, None, None, None, None, None) == m.MOE_OK


def test_block_norm_refusals(lib):
    sh, f = ctypes.byref(m.moe_shape(2, 6, 8, 2, 256, 0)), lib.moe_block_norm
    # x post gate res gamma res_out y q s
    each_pointer(f, (sh, 1e-6, 1.0, 1), 9, optional=(1, 2, 3, 5, 6))
    assert f(sh, 1e-6, 1.0, 1, GOOD, None, None, None, GOOD, *[None] * 4, None) == m.MOE_EINVAL
    for gates in (0, -1, 5, 24):
        assert f(sh, 1e-6, 1.0, gates, *[GOOD] * 9, None) == m.MOE_EINVAL
    for eps, scale in ((-1e-6, 1.0), (float("nan"), 1.0), (float("inf"), 1.0),
                       (1e-6, float("nan")), (1e-6, -float("inf"))):
        assert f(sh, eps, scale, 1, *[GOOD] * 9, None) == m.MOE_EINVAL
    for shape, code in (((2, 4, 8, 2, 200, 0), m.MOE_EINVAL), ((2, -1, 8, 2, 256, 0), m.MOE_EINVAL),
                        ((2, 4, 8, 2, 65664, 0), m.MOE_ENOTSUP)):
        assert f(ctypes.byref(m.moe_shape(*shape)), 1e-6, 1.0, 1, *[GOOD] * 9, None) == code
    assert f(None, 1e-6, 1.0, 1, *[GOOD] * 9, None) == m.MOE_EINVAL
    none = ctypes.byref(m.moe_shape(2, 0, 8, 2, 256, 0))
    assert f(none, 1e-6, 1.0, 3, *[None] * 9, None) == m.MOE_OK


class Device:
    """A device tensor as the binding looks at one."""

    def __init__(self, n, device=0, cuda=True, dtype=torch.bfloat16):
        self.nbytes, self.is_cuda, self.device_, self.dtype = n, cuda, device, dtype

    def get_device(self):
        return self.device_ if self.is_cuda else -1

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


CALLS = {
    "moe_linear": lambda sh, t: m.moe_linear(sh, 64, 64, t["x"], t["w"], t["y"], bias=t["bias"],
                                             res=t["res"], status=t["status"]),
    "moe_linear_glu": lambda sh, t: m.moe_linear_glu(sh, 64, 64, t["x"], t["w13"], t["h"],
                                                     bias=t["bias"], status=t["status"]),
    "moe_topk": lambda sh, t: m.moe_topk(sh, t["logits"], t["topk_idx"], t["topk_w"],
                                         bias=t["bias"]),
    "moe_block_norm": lambda sh, t: m.moe_block_norm(
        sh, t["x"], t["gamma"], 1e-6, res_out=t["res_out"], y=t["y"], q=t["q"], s=t["s"],
        post_gamma=t["post_gamma"], gate=t["gate"], res=t["res"]),
}
# bytes that each call's buffers need for two rows of 64, 4 experts of which 2, H = 256
NEEDS = {
    "moe_linear": dict(x=256, w=8192, y=256, bias=128, res=256, status=4),
    "moe_linear_glu": dict(x=256, w13=16384, h=256, bias=256, status=4),
    "moe_topk": dict(logits=32, topk_idx=16, topk_w=16, bias=16),
    "moe_block_norm": dict(x=1024, gamma=512, res_out=1024, y=1024, q=512, s=16, post_gamma=512,
                           gate=512, res=1024),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_binding_refuses_small_host_and_foreign_tensors(lib, monkeypatch, name):
    sh, launched = m.make_shape(1, 2, 4, 2, 256), []

    class Lib:
        def __getattr__(self, fn):
            return lambda *a: launched.append(fn) or m.MOE_OK
    monkeypatch.setattr(m, "_lib", Lib())
    monkeypatch.setattr(m, "_stream_on", lambda stream, device: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    good = {k: Device(n) for k, n in NEEDS[name].items()}
    CALLS[name](sh, good)
    assert launched == [name]
    for k, n in NEEDS[name].items():
        for bad in (Device(n - 1), Device(n, device=1), Device(n, cuda=False)):
            with pytest.raises(ValueError, match=f"^{k}:"):
                CALLS[name](sh, {**good, k: bad})
    assert launched == [name]


def test_binding_names_and_output_type(lib, monkeypatch):
    sh, seen = m.make_shape(1, 2, 4, 2, 256), []

    class Lib:
        @staticmethod
        def moe_linear(*a):
            seen.append(a)
            return m.MOE_OK
        moe_topk = moe_linear
    monkeypatch.setattr(m, "_lib", Lib)
    monkeypatch.setattr(m, "_stream_on", lambda stream, device: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    big = Device(1 << 16)
    m.moe_linear(sh, 64, 64, big, big, Device(256))
    m.moe_linear(sh, 64, 64, big, big, Device(512, dtype=torch.float32), act="gelu")
    assert seen[0][3] == 0 and seen[0][8] == 0x10000 and seen[0][9] is None
    assert seen[1][3] == 3 and seen[1][8] is None and seen[1][9] == 0x10000
    with pytest.raises(ValueError, match="y"):
        m.moe_linear(sh, 64, 64, big, big, Device(511, dtype=torch.float32))
    with pytest.raises(ValueError, match="act"):
        m.moe_linear(sh, 64, 64, big, big, big, act="swish")
    with pytest.raises(ValueError, match="score"):
        m.moe_topk(sh, big, big, big, score="tanh")
