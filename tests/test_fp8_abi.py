"""The FP8 and routing calls refuse bad arguments before anything is enqueued, and the reference forms
that the GPU tests use are pinned (no device needed)."""
import ctypes

import numpy as np
import pytest

import int4_routed_expert_sigmoid_amd as coli
from tests import fp8_refs as ref

EINVAL, EUNSUP, OK = coli.COLI_EINVAL, coli.COLI_EUNSUPPORTED, coli.COLI_OK


@pytest.fixture(scope="module")
def L():
    return coli.lib()


def test_route_refusals(L):
    def fwd(l=16, dt=0, T=2, E=8, k=2, score=0, groups=2, kept=1, top=2, norm=1, scale=1.0, idx=16, w=16):
        return L.coli_moe_route_groups(l, dt, None, T, E, k, score, groups, kept, top, norm, scale, idx, w, None, None)

    def bwd(l=16, dt=0, T=2, E=8, k=2, score=0, scale=1.0, idx=16, w=16, dl=16, gdt=0):
        return L.coli_moe_route_groups_bwd(w, l, dt, idx, T, E, k, score, 1, scale, None, dl, gdt, None)

    for f in (fwd, bwd):
        assert f(T=-1) == EINVAL and f(E=0) == EINVAL and f(k=0) == EINVAL and f(k=9) == EINVAL
        assert f(E=1025) == EUNSUP and f(E=64, k=33) == EUNSUP and f(T=1 << 26) == EUNSUP
        assert f(dt=3) == EUNSUP and f(dt=-1) == EUNSUP
        assert f(score=2) == EINVAL and f(scale=float("nan")) == EINVAL and f(scale=float("inf")) == EINVAL
        assert f(l=None) == EINVAL and f(idx=None) == EINVAL and f(w=None) == EINVAL
        assert f(T=0, l=None, idx=None, w=None) == OK
    assert fwd(groups=3) == EINVAL and fwd(groups=0) == EINVAL and fwd(E=130, groups=65, kept=65) == EUNSUP
    assert fwd(kept=0) == EINVAL and fwd(kept=3) == EINVAL and fwd(k=5) == EINVAL     # one group of 4 experts
    assert fwd(top=0) == EINVAL and fwd(top=3) == EINVAL
    assert bwd(dl=None) == EINVAL and bwd(gdt=3) == EUNSUP


def test_quantize_refusals(L):
    def rows(x=16, dt=0, r=4, c=64, ld=64, q=16, s=16):
        return L.coli_quantize_fp8(x, dt, r, c, ld, q, s, None)

    def back(x=16, dt=0, r=4, c=64, ld=64, q=16, s=16):
        return L.coli_dequantize_fp8(q, s, r, c, 1, x, dt, ld, None)

    def matrix(x=16, dt=0, r=32, c=64, ld=64, q=16, s=16, n=2, xs=2048, qs=2048, ss=4, qt=None, st=None):
        return L.coli_quantize_fp8_matrix(x, dt, n, r, c, ld, xs, q, qs, s, ss, qt, qs, st, ss, None)

    def columns(x=16, dt=0, r=4, c=64, ld=64, qt=16, st=16, off=16, E=2, P=4, q=None, s=None):
        return L.coli_quantize_fp8_columns(x, dt, r, c, ld, off, E, qt, P, st, q, s, None)

    for f in (rows, back, matrix, columns):
        assert f(c=40) == EINVAL and f(c=0) == EINVAL and f(r=-1) == EINVAL and f(ld=63) == EINVAL
        assert f(dt=3) == EUNSUP and f(dt=-1) == EUNSUP and f(x=None) == EINVAL
        assert f(c=1 << 30, ld=1 << 30) == EUNSUP if f is not columns else True
        assert f(r=0, x=None) == OK
    for f in (rows, back, matrix):
        assert f(q=24) == EINVAL and f(s=18) == EINVAL and f(q=None) == EINVAL and f(s=None) == EINVAL
    assert rows(r=1 << 40) == EUNSUP and back(r=1 << 40) == EUNSUP
    assert L.coli_dequantize_fp8(16, 16, 4, 64, 2, 16, 0, 64, None) == EINVAL

    def many(q=16, qs=2048, s=16, ss=4, n=2, r=20, c=64, x=16, dt=0, ld=64, xs=2048):
        return L.coli_dequantize_fp8_matrix(q, qs, s, ss, n, r, c, x, dt, ld, xs, None)

    assert many(c=40) == EINVAL and many(c=0) == EINVAL and many(r=-1) == EINVAL and many(ld=63) == EINVAL and many(n=-1) == EINVAL
    assert many(dt=3) == EUNSUP and many(r=1 << 30, n=1) == EUNSUP and many(xs=1 << 60) == EUNSUP and many(n=1 << 30) == EUNSUP
    assert many(qs=24) == EINVAL and many(qs=-16) == EINVAL and many(ss=6) == EINVAL and many(ss=-4) == EINVAL
    assert many(xs=20 * 64 - 1) == EINVAL and many(q=24) == EINVAL and many(s=18) == EINVAL
    assert many(q=None) == EINVAL and many(s=None) == EINVAL and many(x=None) == EINVAL
    assert many(n=0, q=None, s=None, x=None) == OK and many(r=0, q=None, s=None, x=None) == OK
    assert matrix(q=None, s=None) == EINVAL                      # no output
    assert matrix(n=-1) == EINVAL and matrix(n=0) == OK
    assert matrix(xs=2047) == EINVAL and matrix(qs=2032) == EINVAL and matrix(ss=0) == EINVAL
    assert matrix(qs=2056) == EINVAL and matrix(ss=6) == EINVAL
    assert matrix(r=24, qt=16, st=16) == EINVAL                  # the transposed rows are no multiple of 16
    assert matrix(qt=24, st=16) == EINVAL and matrix(qt=16) == EINVAL
    assert matrix(r=1 << 30) == EUNSUP and matrix(r=1 << 24, c=1 << 20, ld=1 << 20, n=1) == EUNSUP
    assert columns(P=1) == EINVAL and columns(P=-1) == EINVAL and columns(P=1 << 24) == EUNSUP
    assert columns(E=0) == EINVAL and columns(E=1025, P=1 << 20) == EUNSUP and columns(off=None) == EINVAL
    assert columns(qt=None) == EINVAL and columns(st=None) == EINVAL and columns(qt=24) == EINVAL
    assert columns(q=16) == EINVAL and columns(q=24, s=16) == EINVAL


def test_product_refusals(L):
    def mm(a=16, s=16, rows=4, K=64, off=16, E=2, table=16, q=0, so=256, n=8, y=16, dt=0, ld=8, ws=None):
        return L.coli_fp8_matmul(a, s, rows, K, off, E, table, q, so, n, y, dt, ld, ws, 1 << 20, None)

    def sw(a=16, s=16, rows=4, K=64, off=16, E=2, table=16, q=0, so=256, n=16, y=16, ys=16, dt=0, ld=16, uq=1024, us=512, ws=None):
        return L.coli_fp8_swiglu(a, s, rows, K, off, E, table, q, so, uq, us, n, y, ys, dt, ld, ws, 1 << 20, None)

    for f in (mm, sw):
        assert f(rows=-1) == EINVAL and f(K=40) == EINVAL and f(K=0) == EINVAL and f(K=(1 << 22) + 16) == EUNSUP
        assert f(n=0) == EINVAL and f(E=0) == EINVAL and f(E=1025) == EUNSUP and f(off=None) == EINVAL
        assert f(ld=7) == EINVAL and f(dt=3) == EUNSUP and f(dt=-1) == EUNSUP
        assert f(q=8) == EINVAL and f(so=6) == EINVAL and f(a=24) == EINVAL and f(s=18) == EINVAL
        assert f(a=None) == EINVAL and f(table=None) == EINVAL and f(y=None) == EINVAL and f(s=None) == EINVAL
        assert f(rows=0, a=None, table=None, y=None) == OK
        assert f(n=(1 << 31) - 1, ld=1 << 31) == EUNSUP and f(rows=(1 << 31) - 1) == EUNSUP
    assert mm(ws=24) == EINVAL
    assert mm(dt=coli.FP8) == EUNSUP                             # only the SwiGLU writes FP8
    assert sw(n=24, ld=24, dt=coli.FP8) == EINVAL and sw(dt=coli.FP8, ys=None) == EINVAL and sw(dt=coli.FP8, y=24) == EINVAL
    assert sw(uq=8) == EINVAL and sw(us=2) == EINVAL and sw(dt=coli.FP8, ws=24) == EINVAL

    def wg(g=16, gs=16, x=16, xs=16, P=4, rows=4, off=16, E=2, N=16, K=32, acc=0, dw=16, dt=0, ld=32, ws=None):
        return L.coli_fp8_wgrad(g, gs, x, xs, P, rows, off, E, N, K, acc, dw, dt, ld, ws, 1 << 20, None)

    assert wg(rows=-1) == EINVAL and wg(P=1) == EINVAL and wg(P=-1) == EINVAL and wg(P=1 << 24) == EUNSUP
    assert wg(E=0) == EINVAL and wg(E=1025, P=1 << 20) == EUNSUP and wg(off=None) == EINVAL
    assert wg(N=24) == EINVAL and wg(K=24) == EINVAL and wg(N=0) == EINVAL and wg(K=0) == EINVAL
    assert wg(dt=3) == EUNSUP and wg(ld=31) == EINVAL and wg(ld=1 << 56) == EUNSUP and wg(N=1 << 30) == EUNSUP
    assert wg(dw=None) == EINVAL and wg(g=None) == EINVAL and wg(xs=None) == EINVAL and wg(g=24) == EINVAL
    assert wg(gs=18) == EINVAL and wg(xs=17) == EINVAL and wg(ws=24) == EINVAL
    assert wg(rows=0, acc=1, g=None, gs=None, x=None, xs=None) == OK
    assert L.coli_moe_dispatch_fp8(16, 0, 2, 2, 40, 40, 16, 16, 16, None) == EINVAL
    assert L.coli_moe_dispatch_fp8(16, 0, 2, 2, 32, 31, 16, 16, 16, None) == EINVAL
    assert L.coli_moe_dispatch_fp8(16, 0, 2, 2, 32, 32, 16, 24, 16, None) == EINVAL
    assert L.coli_moe_dispatch_fp8(None, 0, 2, 2, 32, 32, 16, 16, 16, None) == EINVAL
    assert L.coli_moe_dispatch_fp8(None, 0, 0, 2, 32, 32, None, None, None, None) == OK


def test_sizes(L):
    assert coli.fp8_column_blocks(1, 256) == 1 and coli.fp8_column_blocks(128, 1) == 1 and coli.fp8_column_blocks(129, 1) == 2
    assert coli.fp8_column_blocks(0, 4) == 0 and coli.fp8_column_blocks(300, 2) == 4       # 1 + 299 rows
    for rows in (1, 5, 127, 128, 129, 1000):
        for E in (1, 3, 64):
            n = coli.fp8_column_blocks(rows, E)
            assert coli.fp8_column_blocks(coli._rows_of_blocks(n, E), E) <= n and coli._rows_of_blocks(n, E) >= rows
    nb = ctypes.c_size_t()
    size = coli.lib().coli_fp8_swiglu_workspace_size
    for rows, K, E, inter, grouped, want in (  # into FP8
            (8, 6144, 256, 2048, 1, 8 * 2048 * 4), (1, 2064, 1, 144, 0, 144 * 4), (1, 1024, 1, 144, 0, 0), (64, 6144, 40, 2048, 1, 0),
                                             (4096, 6144, 256, 2048, 1, 0), (0, 64, 4, 64, 1, 0)):
        assert size(rows, K, E, inter, grouped, coli.FP8, ctypes.byref(nb)) == OK and nb.value == want
    assert size(8, 6144, 256, 2048, 1, 1, ctypes.byref(nb)) == OK and nb.value == 0
    assert size(256, 6144, 1, 2048, 0, 1, ctypes.byref(nb)) == OK and nb.value == 6 * 256 * 2048 * 2 * 4
    assert size(4, 40, 1, 16, 0, 0, ctypes.byref(nb)) == EINVAL and size(4, 48, 2, 16, 0, 0, ctypes.byref(nb)) == EINVAL
    assert size(4, 48, 1, 16, 0, 0, None) == EINVAL and size(4, 48, 1, 16, 0, 3, ctypes.byref(nb)) == EUNSUP
    size = coli.lib().coli_fp8_matmul_workspace_size
    for rows, K, E, n, dtype, parts in ((8, 8192, 1, 8192, 1, 0), (64, 8192, 1, 8192, 1, 8), (128, 8192, 1, 8192, 1, 6), (8191, 8192, 1, 8192, 0, 0),
                                        (512, 8192, 1, 8192, 0, 2), (16384, 2048, 256, 6144, 1, 0), (0, 64, 1, 64, 0, 0)):
        assert size(rows, K, E, n, int(E > 1), dtype, ctypes.byref(nb)) == OK and nb.value == 4 * parts * rows * n
    assert size(4, 40, 1, 16, 0, 0, ctypes.byref(nb)) == EINVAL and size(4, 48, 2, 16, 0, 0, ctypes.byref(nb)) == EINVAL
    assert size(4, 48, 1, 16, 0, 3, ctypes.byref(nb)) == EUNSUP and size(4, 48, 1, 16, 0, 0, None) == EINVAL
    size = coli.lib().coli_fp8_wgrad_workspace_size
    for rows, E, n, K, parts in ((4095, 1, 6144, 8192, 1), (16384, 64, 2048, 6144, 1), (500, 1, 128, 128, 1), (0, 1, 16, 16, 1),
                                 (4096, 1, 128, 256, 16), (8082, 1, 2384, 1024, 3), (1400, 1, 48, 80, 5),
                                 (4096, 4, 128, 256, 1), (16000, 4, 144, 272, 13)):
        assert size(rows, E, n, K, ctypes.byref(nb)) == OK and nb.value == (parts * E * n * K * 4 if parts > 1 else 0)
    assert size(-1, 1, 16, 16, ctypes.byref(nb)) == EINVAL and size(4, 0, 16, 16, ctypes.byref(nb)) == EINVAL
    assert size(4, 1, 24, 16, ctypes.byref(nb)) == EINVAL and size(4, 1, 16, 0, ctypes.byref(nb)) == EINVAL
    assert size(4, 1, 16, 16, None) == EINVAL and size(4, 1025, 16, 16, ctypes.byref(nb)) == EUNSUP
    off, nbytes = coli.fp8_blob_layout(coli.MoEShape(6144, 2048, 256))
    m, n = 6144 * 2048, 4 * 48 * 16
    assert off == [0, m, 2 * m, 3 * m, 3 * m + n, 3 * m + 2 * n] and nbytes == 3 * (m + n)
    off, nbytes = coli.fp8_blob_layout(coli.MoEShape(32, 64, 1, top_k=1))
    m = 32 * 64
    assert off == [0, m, 2 * m, 3 * m, 3 * m + 256, 3 * m + 512] and nbytes == 3 * m + 768
    with pytest.raises(coli.ColiError):
        coli.fp8_blob_layout(coli.MoEShape(48, 32, 1, top_k=1))


def test_binding_refusals():
    import torch
    x, i = torch.zeros(4, 32), torch.zeros(4, 2, dtype=torch.int32)
    for f in (lambda: coli.quantize_fp8(x), lambda: coli.quantize_fp8_matrix(x), lambda: coli.quantize_fp8_columns(x),
              lambda: coli.route_groups(x, None, 2), lambda: coli.route_groups_bwd(x, x, i), lambda: coli.dispatch_fp8(x, i),
              lambda: coli.dequantize_fp8(x.to(torch.uint8), x), lambda: coli.fp8_matmul(x.to(torch.uint8), x, i, 4),
              lambda: coli.fp8_wgrad(x, x, x, x)):
        with pytest.raises(ValueError, match="device tensor"):
            f()
    with pytest.raises(ValueError, match="score"):
        coli._score("relu")


def test_current_device_without_torchs_inner_call(monkeypatch):
    """The calls find the current device with a torch that lacks the inner function."""
    import torch
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    coli._device_call.cache_clear()
    try:
        assert coli._device_call() is torch.cuda.current_device
    finally:
        coli._device_call.cache_clear()


def test_numbers_that_a_c_int_would_cut():
    """Refused, not taken as their lower 32 (or 64) bits."""
    import torch
    x, far = torch.zeros(4, 32), 2 ** 32
    for how in (dict(groups=far + 2), dict(groups=2, groups_kept=far + 1), dict(group_top=far + 2), dict(groups=2 - far),
                dict(group_top=-far + 1)):
        with pytest.raises(ValueError, match="32 bits"):
            coli.route_groups(x, None, 2, **how)
    with pytest.raises(ValueError, match="32 bits"):
        coli.route_groups(x[:0], None, far + 2)
    with pytest.raises(ValueError, match="32 bits"):
        coli.fp8_column_blocks(far + 5, 1)
    with pytest.raises(ValueError, match="32 bits"):
        coli.fp8_column_blocks(5, far + 1)
    for sizes in ((far + 8, 64, 1, 64), (8, far + 64, 1, 64), (8, 64, far + 1, 64), (8, 64, 1, far + 64)):
        with pytest.raises(ValueError, match="32 bits"):
            coli.debug_fp8_kernel(*sizes, grouped=sizes[2] > 1)
    assert coli.debug_fp8_kernel(64, 8192, 1, 8192, grouped=far) == coli.debug_fp8_kernel(64, 8192, 1, 8192, grouped=True)


def test_reference_codes():
    """The codes against torch's type, the scale rule by its definition."""
    import torch
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.CODES, equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 40001), ref.CODES[:126], (ref.CODES[:126] + ref.CODES[1:127]) / 2])
    assert np.array_equal(ref.encode(x), torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    for top in (448.0, 448.0000305, 447.9, 1.0, 1.75, 1.7500001, 3e-39, 0.0, 3.4e38, 2.0 ** -118 * 1.75, 2.0 ** -118 * 1.76):
        s = ref.scale_value(ref.scale_code(np.float32(top)))
        assert float(np.float32(top)) <= 448 * s and (s == 2.0 ** -126 or float(np.float32(top)) > 224 * s)
    assert ref.scale_code(np.inf) == 255 and ref.scale_code(np.nan) == 255


def test_reference_route_gradient():
    """The formula against central differences of the weights (and scores) for fixed choices."""
    rng = np.random.default_rng(5)
    logits = rng.standard_normal((5, 12))
    logits[1, 3] = -np.inf
    idx = np.stack([rng.permutation(12)[:4] for _ in range(5)]).astype(np.int32)
    idx[2, 3] = -1
    idx[4] = -1
    gw, gs = rng.standard_normal((5, 4)), rng.standard_normal((5, 12))
    for kind in ("sigmoid", "softmax"):
        for norm in (True, False):
            def f(l):
                return (gw * ref.weights(l, idx, kind, norm, 2.5) * (idx >= 0)).sum(1) + (gs * ref.scores(l, kind)).sum(1)
            got = ref.route_grad(gw, logits, idx, kind, norm, 2.5, gs)
            for e in range(12):
                d = np.zeros_like(logits)
                d[:, e] = 1e-5
                diff = (f(logits + d) - f(logits - d)) / 2e-5
                assert np.abs(got[:, e] - diff).max() < 1e-8


def test_cases_reach_every_kernel():
    """The sizes of the products' tests run the kernels that they are named after, SwiGLU's reach all but the first too."""
    from tests.fp8_cases import CASES
    reached = {False: set(), True: set()}
    for kernel, wide, counts, K, N, before, behind in CASES:
        one = isinstance(counts, int)
        rows, E = (counts, 1) if one else (sum(counts) + before + behind, len(counts))
        assert coli.debug_fp8_kernel(rows, K, E, N, grouped=not one) == kernel
        assert coli.debug_fp8_kernel(rows, K, E, N, grouped=not one, wide=True) == wide
        for w in (False, True):
            reached[w].add(coli.debug_fp8_kernel(rows, K, E, N, grouped=not one, swiglu=True, wide=w))
    assert {c[0] for c in CASES} == set(coli.FP8_KERNELS) and {c[1] for c in CASES} == set(coli.FP8_KERNELS[:3])
    assert reached[False] == set(coli.FP8_KERNELS[1:]) and reached[True] == set(coli.FP8_KERNELS[1:3])


def test_cases_reach_every_form_of_fp8_rows():
    """FP8_ROWS reaches the forms that it names, with a K that is a multiple of 512 (scales 16 bytes at a time), one that ends
    after a block and one that ends inside it; what the workspace is for tells the parts."""
    from tests.fp8_cases import FP8_ROWS
    reached = set()
    for form, counts, K, inter, before, behind in FP8_ROWS:
        one = isinstance(counts, int)
        rows, E = (counts, 1) if one else (sum(counts) + before + behind, len(counts))
        exact = rows * inter < 1 << 20
        parts, rest = divmod(coli._fp8_swiglu_ws(rows, K, E, inter, not one, coli.FP8), 8 * rows * inter)
        assert rest == 0 and (form.startswith("exact")) == exact and ("parts" in form) == (parts >= 2)
        if not parts:
            assert coli.debug_fp8_kernel(rows, K, E, inter, grouped=not one, swiglu=True, wide=exact) == "lines_128"
        reached.add((form, "groups" if K % 512 == 0 else "blocks" if K % 128 == 0 else "units"))
    assert reached >= {(f, k) for f in ("exact tiles", "exact parts", "parts") for k in ("groups", "units")} | {("exact tiles", "blocks")}


def test_workspaces_beside_the_named_kernel():
    """debug_fp8_kernel names the kernel without a workspace, `wide` are exact products; the workspace's size tells what runs
    with one: parts of the columns, or (few rows into FP8) f32 rows between two launches."""
    def run(rows, K, E, n, code):
        wide = code == 0 or (code == coli.FP8 and rows * n < 1 << 20)
        ws = (coli._fp8_swiglu_ws if code == coli.FP8 else coli._fp8_matmul_ws)(rows, K, E, n, E > 1, code)
        return coli.debug_fp8_kernel(rows, K, E, n, grouped=E > 1, swiglu=code == coli.FP8, wide=wide), ws // (4 * rows * n)

    assert run(64, 8192, 1, 8192, 1) == ("few_rows_32", 8) and run(256, 6144, 1, 2048, 1)[0] == "few_rows_32"
    assert run(256, 6144, 1, 2048, 1)[1] >= 2 and run(8, 8192, 1, 8192, 1)[1] == 0
    assert run(4, 2048, 4, 640, coli.FP8) == ("few_rows_32", 1)          # two launches
    assert run(127, 8192, 1, 8192, coli.FP8)[1] >= 2 and run(128, 8192, 1, 8192, coli.FP8)[1] >= 2


def test_kernel_choice():
    """The choice follows times measured on both sides (graphs, warm caches; us)."""
    def pick(rows, K, E, N, **how):
        return coli.debug_fp8_kernel(rows, K, E, N, grouped=E > 1, **how)

    assert pick(64, 8192, 1, 8192) == "few_rows_32"                 # 47 against 56
    assert pick(128, 8192, 1, 8192) == "lines_128"                  # 56 against 90
    assert pick(128, 8192, 1, 8192, wide=True) == "few_rows_32"     # 91 against 105
    assert pick(192, 8192, 1, 8192, wide=True) == "lines_128"       # 107 against 134
    assert pick(1024, 8192, 1, 8192) == "lines_128"                 # 72 against 103 for tiles of 256
    assert pick(2048, 8192, 1, 8192) == "lines_256"                 # 121 against 135 for tiles of 128
    assert pick(8192, 8192, 1, 8192) == "lines_256"                 # 453 against 534
    assert pick(256, 2048, 1, 6144) == "lines_128"                  # 20 against 36
    assert pick(256, 6144, 1, 2048) == "few_rows_32"                # 35 against 43
    assert pick(512, 6144, 1, 2048) == "lines_128"                  # 45 against 68
    assert pick(1024, 2048, 64, 2048) == "lines_128"                # 49 against 71
    assert pick(256, 2048, 16, 1024, wide=True) == "few_rows_32"    # 14 against 33
    assert pick(512, 6144, 256, 2048, swiglu=True) == "few_rows_32"     # 928 against 988
    assert pick(2048, 6144, 256, 2048, swiglu=True) == "lines_128"      # 1102 against 1166
    assert pick(1, 16, 1, 1 << 27) == "lines_128"                   # more workgroups than a launch may have
