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


# (experts, N, K, rows an expert, us of few_rows, us of lines of 128 rows), matrices from HBM, one MI355X: the sizes on
# either side of the crossing.
TIMES = [(1, 8192, 8192, 64, 30.5, 40.1), (1, 8192, 8192, 96, 44.1, 42.9), (1, 8192, 8192, 128, 56.9, 46.1),
         (1, 6144, 2048, 128, 12.2, 16.4), (1, 6144, 2048, 192, 17.8, 16.3), (1, 4096, 1024, 256, 8.8, 12.0),
         (1, 4096, 1024, 384, 12.6, 12.1), (1, 2048, 4096, 384, 23.2, 25.0), (1, 2048, 4096, 512, 29.7, 25.0),
         (8, 2048, 2048, 48, 14.2, 15.6), (8, 2048, 2048, 64, 16.7, 16.2), (8, 2048, 2048, 96, 24.4, 17.2),
         (8, 4096, 1024, 32, 10.7, 11.7), (8, 4096, 1024, 48, 14.9, 11.9), (4, 6144, 2048, 32, 14.6, 15.7),
         (4, 6144, 2048, 48, 19.7, 16.0), (32, 1024, 2048, 5, 10.3, 15.7), (32, 1024, 2048, 32, 17.1, 16.5),
         (32, 1024, 2048, 48, 24.5, 16.9), (1, 4096, 6144, 192, 31.0, 36.2), (1, 4096, 6144, 256, 40.0, 37.8),
         (8, 4096, 6144, 5, 25.2, 35.9), (8, 4096, 6144, 17, 43.6, 37.6)]


@pytest.mark.parametrize("E,N,K,per,few,lines", TIMES)
def test_choice_takes_the_kernel_that_measured_faster(E, N, K, per, few, lines):
    want = ("few_rows_4" if K >= 4096 else "few_rows_2") if few < lines else "lines_128"
    assert coli.debug_mxfp4_kernel(E * per, K, E, N, E > 1) == want
