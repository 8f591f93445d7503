"""The MXFP4 and permutation calls refuse bad arguments before anything is
enqueued, and the reference forms the GPU tests use are pinned (no device needed)."""
import ctypes

import numpy as np
import pytest

import int4_routed_expert_sigmoid_amd as coli
from tests import mxfp4_refs as ref

EINVAL, EUNSUP, OK = coli.COLI_EINVAL, coli.COLI_EUNSUPPORTED, coli.COLI_OK


@pytest.fixture(scope="module")
def L():
    return coli.lib()


def test_quantize_refusals(L):
    for f in (lambda x, dt, r, c, ld, q, s: L.coli_quantize_mxfp4(x, dt, r, c, ld, q, s, None),
              lambda x, dt, r, c, ld, q, s: L.coli_dequantize_mxfp4(q, s, r, c, x, dt, ld, None)):
        assert f(16, 0, 4, 48, 64, 16, 16) == EINVAL            # cols not in 32s
        assert f(16, 0, -1, 64, 64, 16, 16) == EINVAL
        assert f(16, 0, 4, 0, 64, 16, 16) == EINVAL
        assert f(16, 0, 4, 64, 63, 16, 16) == EINVAL            # stride below the columns
        assert f(16, 3, 4, 64, 64, 16, 16) == EUNSUP            # MXFP4 is no element type
        assert f(16, -1, 4, 64, 64, 16, 16) == EUNSUP
        assert f(None, 0, 4, 64, 64, 16, 16) == EINVAL
        assert f(16, 0, 4, 64, 64, 24, 16) == EINVAL            # codes off a 16-byte boundary
        assert f(16, 0, 1 << 62, 64, 64, 16, 16) == EUNSUP
        assert f(16, 0, 1 << 31, 2048, 2048, 16, 16) == EUNSUP  # more threads than a launch holds
        assert f(None, 0, 0, 64, 64, None, None) == OK
    assert b"one launch" in L.coli_last_error()


def test_blob_layout(L):
    off, nbytes = coli.mxfp4_blob_layout(coli.MoEShape(6144, 2048, 256))
    assert off == [0, 12582912, 18874368, 19660800] and nbytes == 20054016
    off, nbytes = coli.mxfp4_blob_layout(coli.MoEShape(32, 32, 1, top_k=1))
    assert off == [0, 1024, 1536, 1792] and nbytes == 2048
    with pytest.raises(coli.ColiError):
        coli.mxfp4_blob_layout(coli.MoEShape(48, 32, 1, top_k=1))
    s = coli.MoEShape(64, 32, 4, top_k=1).c()
    assert L.coli_quantize_mxfp4_expert(ctypes.byref(s), 16, 16, None, 0, 16, None) == EINVAL
    assert L.coli_quantize_mxfp4_expert(ctypes.byref(s), 16, 16, 16, 3, 16, None) == EUNSUP
    assert L.coli_quantize_mxfp4_expert(ctypes.byref(s), 16, 16, 16, 0, 8, None) == EINVAL


def test_product_refusals(L):
    def mm(a=16, s=16, rows=4, K=64, off=16, E=2, table=16, q=0, so=256, n=8, y=16, dt=0, ld=8):
        return L.coli_mxfp4_matmul(a, s, rows, K, off, E, table, q, so, n, y, dt, ld, None)

    def sw(a=16, s=16, rows=4, K=64, off=16, E=2, table=16, q=0, so=256, n=32, y=16, ys=16, dt=0, ld=32):
        return L.coli_mxfp4_swiglu(a, s, rows, K, off, E, table, q, so, n, y, ys, dt, ld, None)

    for f in (mm, sw):
        assert f(rows=-1) == EINVAL and f(K=48) == EINVAL and f(K=0) == EINVAL
        assert f(K=(1 << 22) + 32) == EUNSUP
        assert f(n=0) == EINVAL and f(E=0) == EINVAL and f(E=1025) == EUNSUP
        assert f(off=None) == EINVAL                            # several experts need offsets
        assert f(ld=7) == EINVAL and f(dt=4) == EUNSUP and f(dt=-1) == EUNSUP
        assert f(q=8) == EINVAL and f(a=24) == EINVAL
        assert f(a=None) == EINVAL and f(table=None) == EINVAL and f(y=None) == EINVAL and f(s=None) == EINVAL
        assert f(rows=0, a=None, table=None, y=None) == OK
    assert mm(dt=coli.MXFP4) == EUNSUP                          # only the SwiGLU writes MXFP4
    assert mm(rows=2_000_000_000, n=2_000_000_000, ld=2_000_000_000, E=1, off=None) == EUNSUP
    assert sw(n=48) == EINVAL and sw(n=2_000_000_000 // 32 * 32, ld=1 << 31) == EUNSUP
    assert sw(dt=coli.MXFP4, ys=None) == EINVAL and sw(dt=coli.MXFP4, y=24) == EINVAL


def test_permutation_refusals(L):
    calls = {
        "dispatch": lambda T=2, k=2, H=8, dt=0, ld=8, p=16: L.coli_moe_dispatch(p, dt, T, k, H, ld, 16, 16, ld, None),
        "mx": lambda T=2, k=2, H=32, dt=0, ld=64, p=16: L.coli_moe_dispatch_mxfp4(p, dt, T, k, H, ld, 16, 16, 16, None),
        "bwd": lambda T=2, k=2, H=8, dt=0, ld=8, p=16: L.coli_moe_dispatch_bwd(p, dt, ld, T, k, H, 16, 16, dt, ld, None),
        "combine": lambda T=2, k=2, H=8, dt=0, ld=8, p=16: L.coli_moe_combine(p, dt, ld, T, k, H, 16, 16, None, 0, 1.0, 16, dt, ld, None),
        "combine_bwd": lambda T=2, k=2, H=8, dt=0, ld=8, p=16: L.coli_moe_combine_bwd(p, dt, ld, 16, dt, ld, T, k, H, 16, 16, 1.0, 16, ld, 16, None),
    }
    for name, f in calls.items():
        assert f(T=-1) == EINVAL and f(k=0) == EINVAL and f(H=0) == EINVAL, name
        assert f(k=1025) == EUNSUP and f(T=1 << 30, k=2) == EUNSUP, name
        assert f(dt=3) == EUNSUP and f(ld=5) == EINVAL and f(ld=1 << 29) == EUNSUP, name
        assert f(p=None) == EINVAL and f(T=0, p=None) == OK, name
    assert calls["mx"](H=48) == EINVAL
    assert L.coli_moe_combine(16, 0, 8, 2, 2, 8, 16, 16, None, 0, float("inf"), 16, 0, 8, None) == EINVAL
    assert L.coli_moe_combine(16, 0, 8, 2, 2, 8, 16, 16, 16, 4, 1.0, 16, 0, 8, None) == EINVAL
    assert L.coli_moe_combine_bwd(16, 0, 8, 16, 0, 8, 2, 2, 8, 16, 16, float("nan"), 16, 8, 16, None) == EINVAL
    top = 3.4028234663852886e38                                 # the largest finite value is one
    assert L.coli_moe_combine(16, 0, 8, 0, 2, 8, 16, 16, None, 0, top, 16, 0, 8, None) == OK
    assert L.coli_moe_combine_bwd(16, 0, 8, 16, 0, 8, 0, 2, 8, 16, 16, -top, 16, 8, 16, None) == OK
    u = lambda T=2, k=2, E=4, inv=16, ws=1 << 20: L.coli_moe_union_inverse(16, T, k, E, 16, 16, 16, 16, 16, inv, 16, ws, None)
    assert u(T=-1) == EINVAL and u(E=2000) == EUNSUP and u(inv=None) == EINVAL and u(ws=0) == coli.COLI_ENOMEM


def test_binding_refuses_host_and_misshapen_tensors():
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="device"):
        coli.quantize_mxfp4(x)
    with pytest.raises(ValueError, match="device"):
        coli.dispatch(x, torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="device"):
        coli.mxfp4_matmul(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8), x, 8)


def test_reference_quantizer():
    # by hand: largest 5 -> scale 1 (code 127); ties to even codes, saturation, signed zero
    x = np.zeros((1, 64))
    x[0, :12] = [5.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5.0, -0.2, 0.26, 0.0, -0.0]
    x[0, 32:35] = [7.9, 1e-3, np.inf]
    q, s = ref.quantize(x)
    assert s.tolist() == [[127, 255]]
    v = ref.values(q, s)[0]
    assert v[:11].tolist() == [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, -4.0, 0.0, 0.5, 0.0]
    assert (q[0, 4] & 15) == 8 and (q[0, 5] >> 4) == 8          # -0.2 and -0.0 keep their sign
    assert np.isnan(v[32:]).all()
    q, s = ref.quantize(np.full((1, 32), 7.9))
    assert s[0, 0] == 127 and (ref.values(q, s) == 6.0).all()   # saturated
    q, s = ref.quantize(np.full((1, 32), 2.0 ** -130))
    assert s[0, 0] == 0 and (q == 0).all()


class _Device:
    """What the binding looks at of a device tensor, without one (sizes that no test could allocate)."""
    is_cuda = True

    def __init__(self, *shape, dtype=None):
        import torch
        self.shape, self.dtype = shape, dtype or torch.uint8

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def is_contiguous(self):
        return True

    def stride(self):
        return tuple(int(np.prod(self.shape[i + 1:], dtype=object)) for i in range(self.dim()))

    def data_ptr(self):
        return 16

    def new_empty(self, shape, dtype=None):
        return _Device(*shape, dtype=dtype)


def test_binding_refuses_sizes_that_the_c_types_would_cut(monkeypatch):
    """A size of 2^32 + n would arrive as n, pass the library's checks and give the product of a part."""
    import torch

    def reached(*args):
        raise AssertionError("the call went on to the library")

    monkeypatch.setattr(coli, "_enqueue", reached)
    K = 2 ** 32 + 32
    one = _Device(1, dtype=torch.int64)
    for a, a_s, table in ((_Device(1, K // 2), _Device(1, K // 32), one),
                          (_Device(1, 16), _Device(1, 1), _Device(2 ** 32 + 1, dtype=torch.int64))):
        with pytest.raises(ValueError, match="2\\^31"):
            coli.mxfp4_matmul(a, a_s, table, 8)
        with pytest.raises(ValueError, match="2\\^31"):
            coli.mxfp4_swiglu(a, a_s, table, 32)
        with pytest.raises(ValueError, match="2\\^31"):
            coli.mxfp4_swiglu(a, a_s, table, 32, dtype="mxfp4")
    with pytest.raises(ValueError, match="2\\^31"):
        coli.union_inverse(_Device(1, 2, dtype=torch.int32), 2 ** 32 + 4)
    with pytest.raises(AssertionError, match="library"):         # the largest K that the library takes is not refused
        coli.mxfp4_matmul(_Device(1, 2 ** 21), _Device(1, 2 ** 17), one, 8)


@pytest.mark.parametrize("kw", [dict(group=64), dict(group=48), dict(topp=-1.0), dict(topp=float("nan")), dict(wbits=3),
                                dict(routed_scale=float("inf")), dict(routed_scale=float("nan"))])
def test_mxfp4_blobs_take_no_account_of_fields_they_do_not_use(L, kw):
    want = coli.mxfp4_blob_layout(coli.MoEShape(96, 32, 4, top_k=2))
    shape = coli.MoEShape(96, 32, 4, top_k=2, **kw)
    assert coli.mxfp4_blob_layout(shape) == want
    s = shape.c()                                               # past the shape, to the pointers' check
    assert L.coli_quantize_mxfp4_expert(ctypes.byref(s), None, 16, 16, 0, 16, None) == EINVAL
    assert b"NULL" in L.coli_last_error()
