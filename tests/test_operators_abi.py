"""Refusals of the norm, the experts' products and the few-token layer: on the
host, before anything touches CUDA."""
from __future__ import annotations

import ctypes

import pytest
import torch

from combine_expert_count_gb300 import moeroute as m

GOOD, BAD, NULL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004), None


@pytest.fixture(scope="module")
def lib():
    from combine_expert_count_gb300 import build
    build.build()
    return m.lib()


def each_pointer(fn, head, n, optional=()):
    """fn(*head, n pointers, NULL) with one pointer at a time misaligned or null."""
    for i in range(n):
        for p in (BAD, NULL):
            if p is NULL and i in optional:
                continue
            args = [GOOD] * n
            args[i] = p
            assert fn(*head, *args, None) == m.MOE_EINVAL, (fn.__name__, i, p)


def test_norm_refusals(lib):
    sh = ctypes.byref(m.moe_shape(2, 4, 8, 2, 256, 0))
    f = lib.moe_rmsnorm
    each_pointer(f, (sh, 1e-6), 7, optional=(1, 3, 4))  # x res gamma res_out y q s
    assert f(sh, 1e-6, GOOD, None, GOOD, None, None, None, None, None) == m.MOE_EINVAL
    for eps in (-1e-6, float("nan"), float("inf")):
        assert f(sh, eps, *[GOOD] * 7, None) == m.MOE_EINVAL
    for shape, code in (((2, 4, 8, 2, 200, 0), m.MOE_EINVAL), ((2, -1, 8, 2, 256, 0), m.MOE_EINVAL),
                        ((2, 4, 8, 2, 65664, 0), m.MOE_ENOTSUP)):
        assert f(ctypes.byref(m.moe_shape(*shape)), 1e-6, *[GOOD] * 7, None) == code
    assert f(None, 1e-6, *[GOOD] * 7, None) == m.MOE_EINVAL


def test_product_refusals(lib):
    sh = ctypes.byref(m.moe_shape(2, 4, 8, 2, 256, 0))
    for f, n in ((lib.moe_expert_gemm, 7), (lib.moe_expert_gemm_swiglu, 8)):
        each_pointer(f, (sh, 256, 256), n, optional=(n - 1,))  # grp_off has to be: E != N
        for width, code in ((0, m.MOE_EINVAL), (-128, m.MOE_EINVAL), (100, m.MOE_EINVAL),
                            (65536 + 128, m.MOE_ENOTSUP)):
            assert f(sh, width, 256, *[GOOD] * n, None) == code
            assert f(sh, 256, width, *[GOOD] * n, None) == code
        assert f(None, 256, 256, *[GOOD] * n, None) == m.MOE_EINVAL
        bad = ctypes.byref(m.moe_shape(3, 4, 8, 2, 256, 0))
        assert f(bad, 256, 256, *[GOOD] * n, None) == m.MOE_EINVAL
        # no rows at all: nothing to do, whatever the row buffers are
        none = ctypes.byref(m.moe_shape(2, 0, 8, 2, 256, 0))
        args = [None] * n
        args[2], args[3], args[4] = GOOD, GOOD, GOOD  # offsets and weights
        assert f(none, 256, 256, *args, None) == m.MOE_OK
    # the up weights make 2 * inter outputs: 65536 of them at most
    assert lib.moe_expert_gemm_swiglu(sh, 32768 + 128, 256, *[GOOD] * 8, None) == m.MOE_ENOTSUP


def test_few_refusals(lib):
    f = lib.moe_layer_few
    sh = ctypes.byref(m.moe_shape(2, 4, 8, 2, 256, 0))
    each_pointer(f, (sh, 256), 11)
    for width, code in ((0, m.MOE_EINVAL), (130, m.MOE_EINVAL), (65536 + 128, m.MOE_ENOTSUP)):
        assert f(sh, width, *[GOOD] * 11, None) == code
    many = ctypes.byref(m.moe_shape(5, 13, 10, 2, 256, 0))
    assert f(many, 256, *[GOOD] * 11, None) == m.MOE_ENOTSUP
    assert f(None, 256, *[GOOD] * 11, None) == m.MOE_EINVAL


def test_binding_checks_sizes(lib):
    sh = m.make_shape(1, 2, 4, 2, 256)
    t = torch.zeros(8)
    with pytest.raises(ValueError):
        m.moe_rmsnorm(sh, t, t, 1e-6, y=t)
    with pytest.raises(ValueError):
        m.moe_expert_gemm(sh, 256, 256, t, t, t, t, t, t)
    with pytest.raises(ValueError):
        m.moe_expert_gemm_swiglu(sh, 256, 256, t, t, t, t, t, t, t)
    with pytest.raises(ValueError):
        m.moe_layer_few(sh, 256, *[t] * 11)
