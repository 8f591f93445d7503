"""The rule that chooses a kernel for an MXFP4 product (no device needed)."""
import ctypes

import pytest

import int4_routed_expert_sigmoid_amd as coli
from tests import mxfp4_cases as cases


@pytest.mark.parametrize("kernel,counts,K,aligned,spare", cases.CASES)
@pytest.mark.parametrize("swiglu", [False, True])
def test_cases_reach_the_kernel_they_name(kernel, counts, K, aligned, spare, swiglu):
    n = cases.matrix_rows(kernel, counts, swiglu)
    assert cases.chosen(coli, counts, spare, K, 2 * n if swiglu else n, aligned) == kernel


def test_every_kernel_has_cases_and_layers():
    assert {c[0] for c in cases.CASES} == set(coli.MXFP4_KERNELS)
    assert {k for l in cases.LAYERS for k in l[5:]} == set(coli.MXFP4_KERNELS)
    for T, E, k, H, I, up, down in cases.LAYERS:
        assert coli.debug_mxfp4_kernel(T * k, H, E, 2 * I) == up and coli.debug_mxfp4_kernel(T * k, I, E, H) == down


def test_refusals():
    L = coli.lib()
    out = ctypes.c_int32(-1)
    ask = lambda rows=4, K=64, E=2, N=8, grouped=1, p=ctypes.byref(out): L.coli_debug_mxfp4_kernel(rows, K, E, N, grouped, 1, p)
    assert ask() == coli.COLI_OK and out.value == 0
    for kw in (dict(rows=0), dict(K=48), dict(K=0), dict(E=0), dict(N=0), dict(grouped=0), dict(p=None)):
        assert ask(**kw) == coli.COLI_EINVAL, kw
