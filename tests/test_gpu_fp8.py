"""FP8 quantisers, grouped products and their gradients against plain 64-bit forms.

Tolerances: the quantisers and their inverse are exact. Products: product_bound's argument for every value and norm_bound's
for all together (fp8_refs), plus half a step of the output type. SwiGLU: the errors of both sums through the derivatives
(|silu'| <= 1.1), 16 half-steps of f32 for exp, divide and the two products, plus the output's half step."""
import numpy as np
import pytest

from tests import fp8_refs as ref
from tests.fp8_cases import CASES, FP8_ROWS

pytestmark = pytest.mark.gpu
DTYPES = ("float32", "bfloat16", "float16")


@pytest.fixture(scope="module")
def coli():
    import int4_routed_expert_sigmoid_amd as c
    c.lib()
    return c


def _dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


def _t(name):
    import torch
    return getattr(torch, name)


def _half_step(name):
    import torch
    return torch.finfo(_t(name)).eps / 2


def _rounding(name, y):
    """Half a step of the type at y: relative to the value, and below the smallest normal number half of the fixed step that
    subnormal numbers have (float16: 2^-25 below 2^-14)."""
    import torch
    return np.maximum(_half_step(name) * np.abs(y), torch.finfo(_t(name)).tiny * _half_step(name))


def _within(err, tol):
    return err.size == 0 or bool((err <= tol).all())


def _host(t):
    return t.double().cpu().numpy()


def _hard(rng, rows, cols):
    """Normal values of very different sizes, with ties between codes, exact ends of ranges, zeros and outliers."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-8, 9, (rows, -(-cols // 16)))).repeat(16, 1)[:, :cols]
    mid = (ref.CODES[:126] + ref.CODES[1:127]) / 2
    ties = rng.choice(np.concatenate([mid, ref.CODES[:127]]), (rows, cols)) * rng.choice([-1.0, 1.0], (rows, cols))
    pick = rng.random((rows, -(-cols // 128))).repeat(128, 1)[:, :cols] < 0.4
    scale = np.exp2(rng.integers(-4, 4, (rows, -(-cols // 128)))).repeat(128, 1)[:, :cols]
    x = np.where(pick, ties * scale, x)
    x[rng.random((rows, cols)) < 0.05] = -0.0
    x[rng.random((rows, cols)) < 0.05] = 0.0
    x[rng.random(rows) < 0.1] = 0.0
    return x


# ---------------------------------------------------------------- quantisers
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,pad", [(1, 16, 0), (1, 128, 0), (3, 144, 0), (1, 6144, 0), (37, 2080, 0), (37, 2080, 5),
                                           (1029, 1040, 0), (513, 2048, 8), (5, 240, 1)])
def test_quantize_rows(coli, dtype, rows, cols, pad):
    import torch
    rng = np.random.default_rng(rows * 1000 + cols + pad)
    full = torch.from_numpy(_hard(rng, rows, cols)).to(_t(dtype))
    buf = torch.full((rows, cols + pad), float("nan"), dtype=_t(dtype))
    buf[:, :cols] = full
    q, s = coli.quantize_fp8(buf.to("cuda")[:, :cols])
    qr, sr = ref.quantize_rows(_host(full))
    assert np.array_equal(_host(s), ref.scale_value(sr))
    assert np.array_equal(q.cpu().numpy(), qr)
    for out in DTYPES:
        out_buf = torch.full((rows, cols + pad), 7.0, dtype=_t(out), device="cuda")
        v = coli.dequantize_fp8(q, s, out=out_buf[:, :cols])
        assert torch.equal(v.cpu(), torch.from_numpy(ref.values(qr, ref.scale_value(sr))).to(_t(out)))
        assert bool((out_buf[:, cols:] == 7.0).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_extremes(coli, dtype):
    """Infinities, NaN, a type's largest and smallest values, every scale border, empty input, rows off a 16-byte boundary."""
    import torch
    info = torch.finfo(_t(dtype))
    x = torch.zeros(10, 256, dtype=_t(dtype))
    x[0, 3], x[0, 133] = float("inf"), float("-inf")
    x[1, 31], x[1, 140] = float("nan"), 1.0
    x[2], x[3] = info.max, info.min
    x[4] = info.tiny
    x[5, :32] = info.smallest_normal * info.eps                  # subnormal
    x[6, 0], x[6, 1] = info.max, info.tiny
    x[7, 0] = info.tiny / 4
    x[8, 0], x[8, 130] = 448.0, 448.0 * (1 + info.eps)            # the largest of one scale, the smallest of the next
    x[9, :128] = torch.linspace(-448, 448, 128)
    q, s = coli.quantize_fp8(x.to("cuda"))
    qr, sr = ref.quantize_rows(_host(x))
    assert np.array_equal(_host(s), ref.scale_value(sr), equal_nan=True) and np.array_equal(q.cpu().numpy(), qr)
    assert sr[0].tolist() == [255, 255] and sr[1, 0] == 255 and sr[1, 1] != 255 and sr[8].tolist() == [127, 128]
    v = coli.dequantize_fp8(q, s)
    assert np.array_equal(_host(v), ref.values(qr, ref.scale_value(sr)).astype(np.float32), equal_nan=True)
    buf = torch.zeros(10 * 256 + 1, dtype=_t(dtype), device="cuda")
    odd = buf[1:].view(10, 256)
    odd.copy_(x)
    q2, s2 = coli.quantize_fp8(odd)
    assert torch.equal(q2, q) and torch.equal(s2.nan_to_num(7.0), s.nan_to_num(7.0))
    q0, s0 = coli.quantize_fp8(torch.empty(0, 64, dtype=_t(dtype), device="cuda"))
    assert q0.shape == (0, 64) and s0.shape == (0, 1) and coli.dequantize_fp8(q0, s0).shape == (0, 64)


def test_all_codes_and_any_scale(coli):
    """Every code under scales that are no powers of two, 0, NaN and infinity, of rows and of matrices."""
    import torch
    q = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(130, 1)
    for s in (torch.rand(130, 2, device="cuda") * 3, torch.rand(2, 2, device="cuda")):
        s[1, 1], s[0, 1] = float("inf"), 0.0
        block = 1 if s.shape[0] == 130 else 128
        with np.errstate(invalid="ignore"):
            want = ref.values(q.cpu().numpy(), _host(s), block).astype(np.float32)
        for out in DTYPES:
            got = coli.dequantize_fp8(q, s, dtype=_t(out)).cpu()
            assert torch.equal(got.nan_to_num(9.0), torch.from_numpy(want).to(_t(out)).nan_to_num(9.0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("count,rows,cols,pad", [(1, 16, 16, 0), (1, 128, 128, 0), (3, 144, 272, 0), (2, 256, 128, 3), (1, 1040, 96, 0),
                                                 (5, 48, 384, 16)])
def test_quantize_matrix(coli, dtype, count, rows, cols, pad):
    import torch
    rng = np.random.default_rng(count * 1000 + rows + cols + pad)
    x = torch.from_numpy(np.stack([_hard(rng, rows, cols) for _ in range(count)])).to(_t(dtype))
    buf = torch.full((count, rows + 1, cols + pad), float("nan"), dtype=_t(dtype), device="cuda")
    buf[:, :rows, :cols] = x.cuda()
    arena = torch.full((count, 3 * rows * cols + 512), 9, dtype=torch.uint8, device="cuda")
    half, nb, nk = rows * cols, -(-rows // 128), -(-cols // 128)
    places = dict(q=arena[:, :half].unflatten(1, (rows, cols)), qt=arena[:, half:2 * half].unflatten(1, (cols, rows)),
                  s=arena[:, 2 * half:2 * half + 4 * nb * nk].view(torch.float32).unflatten(1, (nb, nk)))
    for given in ({}, places):
        q, s, qt, st = coli.quantize_fp8_matrix(buf[:, :rows, :cols], transposed=True, **given)
        for i in range(count):
            qr, sr = ref.quantize_matrix(_host(x[i]))
            assert np.array_equal(q[i].cpu().numpy(), qr) and np.array_equal(_host(s[i]), ref.scale_value(sr))
            assert np.array_equal(qt[i].cpu().numpy(), qr.T) and np.array_equal(_host(st[i]), ref.scale_value(sr).T)
    assert bool((arena[:, 2 * half + 4 * nb * nk:] == 9).all())
    one = coli.quantize_fp8_matrix(x[0].cuda())
    assert len(one) == 2 and torch.equal(one[0], q[0]) and torch.equal(one[1], s[0])
    v = coli.dequantize_fp8(q, s)
    assert np.array_equal(_host(v[-1]), ref.values(q[-1].cpu().numpy(), _host(s[-1]), 128))
    for a, b in ((q, s), (qt, st), (places["q"], places["s"])):      # dense, transposed, in buffers with gaps
        back = torch.full((count, a.shape[1] + 1, a.shape[2] + 5), 9.0, dtype=_t(dtype), device="cuda")
        coli.dequantize_fp8(a, b, out=back[:, :-1, :-5])
        for i in range(count):
            want = torch.from_numpy(ref.values(a[i].cpu().numpy(), _host(b[i]), 128)).float().to(_t(dtype))
            assert torch.equal(back[i, :-1, :-5].cpu().nan_to_num(7.0), want.nan_to_num(7.0))
        assert bool((back[:, -1] == 9).all()) and bool((back[..., -5:] == 9).all())
    one = coli.quantize_fp8_matrix(torch.full((20, 32), float("inf"), device="cuda"))   # rows in no 16s: one way round
    assert bool(one[1].isnan().all()) and int(one[0].sum()) == 0


COUNTS = [[1], [0, 3, 0], [128, 129, 0, 1, 127, 256], [7] * 70, [0] * 5, [300], [0, 0, 500, 12]]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(COUNTS)))
def test_quantize_columns(coli, dtype, case):
    import torch
    counts, cols = COUNTS[case], (16, 144, 272, 128, 32, 400, 96)[case]
    rng = np.random.default_rng(case)
    before, behind = (0, 3)[case % 2], (0, 0, 5)[case % 3]
    off = np.concatenate([[before], before + np.cumsum(counts)]).astype(np.int32)
    rows = int(off[-1]) + behind
    x = torch.from_numpy(_hard(rng, rows, cols)).to(_t(dtype)) if rows else torch.zeros(0, cols, dtype=_t(dtype))
    if rows > 4:
        x[before, 3] = float("nan")
    want_q, want_s = ref.quantize_columns(_host(x), off)
    B = coli.fp8_column_blocks(rows, len(counts)) + 1
    qt = torch.full((B, cols, 128), 77, dtype=torch.uint8, device="cuda")
    st = torch.full((B, cols), 77, dtype=torch.uint8, device="cuda")
    q = torch.full((rows, cols), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, -(-cols // 128)), 77.0, device="cuda")
    buf = torch.full((rows, cols + 3), 1.0, dtype=_t(dtype), device="cuda")
    buf[:, :cols] = x.cuda()
    coli.quantize_fp8_columns(buf[:, :cols], _dev(off), qt=qt, st=st, q=q, s=s)
    n = len(want_q)
    assert np.array_equal(qt.cpu().numpy()[:n], want_q) and bool((qt[n:] == 77).all())
    assert np.array_equal(st.cpu().numpy()[:n], want_s) and bool((st[n:] == 77).all())
    lo, hi = before, int(off[-1])
    if hi > lo:
        qr, sr = ref.quantize_rows(_host(x[lo:hi]))
        assert np.array_equal(q[lo:hi].cpu().numpy(), qr) and np.array_equal(_host(s[lo:hi]), ref.scale_value(sr), equal_nan=True)
    assert bool((q[:lo] == 77).all()) and bool((q[hi:] == 77).all()) and bool((s[hi:] == 77.0).all())
    if len(counts) == 1 and before + behind == 0:
        a, b = coli.quantize_fp8_columns(x.cuda())
        assert len(a) == -(-rows // 128) and np.array_equal(a.cpu().numpy(), want_q) and np.array_equal(b.cpu().numpy(), want_s)


@pytest.mark.parametrize("dtype", DTYPES)
def test_dispatch(coli, dtype):
    """A token's codes and scales in all of its rows, rows of no slot left as they are."""
    import torch
    rng = np.random.default_rng(2)
    for T, k, H in ((1, 1, 16), (9, 4, 272), (70, 8, 2064), (3, 2, 6144)):
        x = torch.from_numpy(_hard(rng, T, H)).to(_t(dtype))
        inv = rng.permutation(T * k).reshape(T, k).astype(np.int32)
        gone = rng.random((T, k)) < 0.3
        want_q, want_s = ref.quantize_rows(_host(x))
        q = torch.full((T * k, H), 7, dtype=torch.uint8, device="cuda")
        s = torch.full((T * k, -(-H // 128)), 7.0, device="cuda")
        coli.dispatch_fp8(x.cuda(), _dev(np.where(gone, rng.choice([-1, T * k], (T, k)), inv).astype(np.int32)), q=q, s=s)
        for t in range(T):
            for j in range(k):
                p = inv[t, j]
                if gone[t, j]:
                    assert bool((q[p] == 7).all()) and bool((s[p] == 7.0).all())
                else:
                    assert np.array_equal(q[p].cpu().numpy(), want_q[t]) and np.array_equal(_host(s[p]), ref.scale_value(want_s[t]))


def test_quantize_past_32_bits(coli):
    import torch
    rows, cols = 1 << 18, 8208                                    # 2.15e9 bf16 values
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1, -16:] = 3.0
    x[rows // 2, 128] = -1.0
    for src in (x, x[:, :8192]):
        q, s = coli.quantize_fp8(src)
        assert int((q != 0).sum()) == (17 if src is x else 1) and q[rows // 2, 128].item() == 0xF8
        v = coli.dequantize_fp8(q, s, dtype=torch.bfloat16)
        assert v[rows // 2, 128].item() == -1.0 and (src is not x or bool((v[-1, -16:] == 3.0).all()))
        del q, s, v
    q, s, qt, st = coli.quantize_fp8_matrix(x, transposed=True)
    assert q[-1, -1].item() == qt[-1, -1].item() == 0x7C and int((qt != 0).sum()) == 17 and st[-1, -1] == s[-1, -1]
    del q, s
    a, b = coli.quantize_fp8_columns(x)
    assert int((a != 0).sum()) == 17 and a[-1, -1, -1].item() == 0x7C and a[rows // 256, 128, 0].item() == 0xF8
    assert b[-1, -1].item() == 120


# ---------------------------------------------------------------- products
# (Their 64-bit forms are elementary torch operations on the device: sizes that reach every kernel are large for numpy.)
def _codes(rng, *shape):
    """Codes of normal values near the end of the range, as a block's quantised ones are."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 31)))
    x = 110 * torch.randn(*shape, device="cuda", generator=g)
    return x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(q, s, block_rows=1):
    import torch
    v = torch.from_numpy(ref.CODES).cuda()[q.long()]
    s = s.double().repeat_interleave(128, -1)[..., :q.shape[-1]]
    return v * (s if block_rows == 1 else s.repeat_interleave(128, -2)[..., :q.shape[-2], :])


def _scales(rng, mean, *shape):
    import torch
    g = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 31)))
    return mean * (0.5 + torch.rand(*shape, device="cuda", generator=g))


def _weights(rng, E, n, K, parts=1, odd=4):
    """Blobs of `parts` FP8 matrices each with any scales, 16 bytes of something before them; (blobs, table, a function of the
    matrix' values, offsets). odd: where the scales lie behind a multiple of 16 bytes."""
    import torch
    nb, nk = -(-n // 128), -(-K // 128)
    s_off = 16 + parts * n * K + odd
    size = -(-(s_off + 4 * parts * nb * nk) // 16) * 16
    blobs = torch.full((E, size), 0x7F, dtype=torch.uint8, device="cuda")    # NaN wherever a product should not read
    q, s = _codes(rng, E, parts, n, K), _scales(rng, 2e-3, E, parts, nb, nk)
    blobs[:, 16:16 + parts * n * K] = q.flatten(1)
    blobs[:, s_off:s_off + 4 * parts * nb * nk] = s.flatten(1).view(torch.uint8)
    table = blobs.data_ptr() + size * torch.arange(E, dtype=torch.int64)
    return blobs, table.cuda(), lambda e, p=0: _values(q[e, p], s[e, p], 128), dict(q_off=16, s_off=s_off)


def _rows(rng, rows, K, mean=0.01):
    q, s = _codes(rng, rows, K), _scales(rng, mean, rows, -(-K // 128))
    return q, s, _values(q, s)


def _product(a, matrix, off, n, p=0):
    """(y, sum of |terms|) [rows][n]; rows outside the offsets are 0."""
    y = a.new_zeros(a.shape[0], n)
    t = a.new_zeros(a.shape[0], n)
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        if hi > lo:
            m = matrix(e, p).t().contiguous()
            y[lo:hi], t[lo:hi] = a[lo:hi] @ m, a[lo:hi].abs() @ m.abs()
    return y, t


def _groups(counts, before, behind):
    if isinstance(counts, int):
        return None, np.array([0, counts]), counts
    off = np.concatenate([[before], before + np.cumsum(counts)]).astype(np.int32)
    return _dev(off), off, int(off[-1]) + behind


def _case_id(c):
    return f"{c[0]}-{c[2] if isinstance(c[2], int) else len(c[2])}-{c[3]}-{c[4]}"


def _half(dtype, y):
    """_rounding of a tensor."""
    import torch
    return (_half_step(dtype) * y.abs()).clamp_min(torch.finfo(_t(dtype)).tiny * _half_step(dtype))


@pytest.mark.parametrize("odd", (0, 4))                             # (0: scales come 16 bytes at a time)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", CASES, ids=_case_id)
def test_matmul(coli, case, dtype, odd):
    import torch
    kernel, wide, counts, K, n, before, behind = case
    offsets, off, rows = _groups(counts, before, behind)
    E, exact = len(off) - 1, dtype == "float32"
    assert coli.debug_fp8_kernel(rows, K, E, n, grouped=offsets is not None, wide=exact) == (wide if exact else kernel)
    assert coli._fp8_matmul_ws(rows, K, E, n, offsets is not None, 0 if exact else 1) == 0
    rng = np.random.default_rng(K + n)
    _keep, table, matrix, at = _weights(rng, E, n, K, odd=odd)
    a, a_s, va = _rows(rng, rows, K)
    out = torch.full((rows, n + 3), 7.0, dtype=_t(dtype), device="cuda")
    coli.fp8_matmul(a, a_s, table, n, offsets=offsets, out=out[:, :n], **at)
    y, terms = _product(va, matrix, off, n)
    lo, hi = int(off[0]), int(off[-1])
    assert bool((out[:, n:] == 7.0).all()) and bool((out[:lo] == 7.0).all()) and bool((out[hi:] == 7.0).all())
    err, y = (out[lo:hi, :n].double() - y[lo:hi]).abs(), y[lo:hi]
    assert bool((err <= ref.product_bound(K, terms[lo:hi], exact) * (1 + _half_step(dtype)) + _half(dtype, y)).all())
    assert float(err.norm()) <= (ref.norm_bound(K, exact) + _half_step(dtype)) * float(y.norm())
    again = coli.fp8_matmul(a, a_s, table, n, offsets=offsets, dtype=_t(dtype), **at)
    assert torch.equal(again[lo:hi], out[lo:hi, :n])


def _scale_of(top):
    """The quantiser's scale for a block whose largest is `top` (64 bits)."""
    import torch
    return torch.from_numpy(ref.scale_value(ref.scale_code(top.cpu().numpy()))).cuda()


# SwiGLU's columns summed in parts, gate's and up's apart
PARTS = [("", "", 150, 5136, 2051, 0, 0), ("", "", [130, 0, 123], 8192, 528, 3, 4), ("", "", 64, 8192, 8192, 0, 0)]


@pytest.mark.parametrize("odd", (0, 4))
@pytest.mark.parametrize("dtype", DTYPES + ("fp8",))
@pytest.mark.parametrize("case", CASES + PARTS, ids=_case_id)
def test_swiglu(coli, case, dtype, odd):
    import torch
    _, _, counts, K, n, before, behind = case
    n = -(-n // 16) * 16 if dtype == "fp8" else n
    offsets, off, rows = _groups(counts, before, behind)
    E, exact = len(off) - 1, dtype == "float32" or (dtype == "fp8" and rows * n < 1 << 20)      # (below it, codes of exact products)
    code = {"float32": 0, "bfloat16": 1, "float16": 2, "fp8": coli.FP8}[dtype]
    assert case not in PARTS or (exact and E > 1) or coli._fp8_swiglu_ws(rows, K, E, n, offsets is not None, code) >= 2 * 8 * rows * n
    rng = np.random.default_rng(K + n + 1)
    _keep, table, matrix, at = _weights(rng, E, n, K, parts=2, odd=odd)
    a, a_s, va = _rows(rng, rows, K, 0.08 / np.sqrt(K))
    g, tg = _product(va, matrix, off, n, 0)
    u, tu = _product(va, matrix, off, n, 1)
    eg, eu = ref.product_bound(K, tg, exact), ref.product_bound(K, tu, exact)
    silu = g / (1 + torch.exp(-g))
    h = silu * u
    err = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + 16 * 2.0 ** -24 * h.abs()
    lo, hi = int(off[0]), int(off[-1])
    if dtype != "fp8":
        out = torch.full((rows, n + 3), 7.0, dtype=_t(dtype), device="cuda")
        coli.fp8_swiglu(a, a_s, table, n, offsets=offsets, out=out[:, :n], **at)
        assert bool((out[:, n:] == 7.0).all()) and bool((out[:lo] == 7.0).all()) and bool((out[hi:] == 7.0).all())
        assert bool(((out[:, :n].double() - h).abs() <= err * (1 + _half_step(dtype)) + _half(dtype, h))[lo:hi].all())
        return
    new = coli.fp8_swiglu(a, a_s, table, n, offsets=offsets, dtype="fp8", **at)
    up = (at["q_off"] + n * K, at["s_off"] + 4 * -(-n // 128) * -(-K // 128))
    for workspace in (True, False):                               # without the one that few rows may use: one launch, sums in another order
        q = torch.full((rows, n), 77, dtype=torch.uint8, device="cuda")
        s = torch.full((rows, -(-n // 128)), 77.0, device="cuda")
        if workspace:
            coli.fp8_swiglu(a, a_s, table, n, offsets=offsets, out=(q, s), **at)
            assert torch.equal(new[0][lo:hi], q[lo:hi]) and torch.equal(new[1][lo:hi], s[lo:hi])
        elif rows:
            assert coli.lib().coli_fp8_swiglu(a.data_ptr(), a_s.data_ptr(), rows, K, None if offsets is None else offsets.data_ptr(), E,
                                              table.data_ptr(), at["q_off"], at["s_off"], *up, n, q.data_ptr(), s.data_ptr(), coli.FP8,
                                              n, None, 0, coli._stream()) == 0
        assert bool((q[:lo] == 77).all()) and bool((q[hi:] == 77).all()) and bool((s[:lo] == 77.0).all()) and bool((s[hi:] == 77.0).all())
        for b in range(s.shape[1] if hi > lo else 0):
            part, e = h[lo:hi, b * 128:(b + 1) * 128].abs(), err[lo:hi, b * 128:(b + 1) * 128]
            sb = s[lo:hi, b].double()
            assert bool((_scale_of((part - e).clamp_min(0).amax(1)) <= sb).all()) and bool((sb <= _scale_of((part + e).amax(1))).all())
        step = torch.maximum(2.0 ** -4 * (h.abs() + err), 2.0 ** -10 * s.double().repeat_interleave(128, 1)[:, :n])
        assert bool(((_values(q, s) - h).abs() <= err + step)[lo:hi].all())


@pytest.mark.parametrize("odd", (0, 4))
@pytest.mark.parametrize("case", FP8_ROWS, ids=lambda c: f"{c[0].replace(' ', '_')}-{c[2]}-{c[3]}")
def test_swiglu_forms_of_fp8_rows(coli, case, odd):
    test_swiglu(coli, ("", "", *case[1:]), "fp8", odd)


def test_separate_gate_and_up(coli):
    """Gate and up anywhere in the buffer: up before gate, scales before codes."""
    import torch
    rng = np.random.default_rng(8)
    K, n = 272, 48
    a, a_s, _ = _rows(rng, 3, K)
    keep, table, _, at = _weights(rng, 1, n, K, parts=2)
    want = coli.fp8_swiglu(a, a_s, table, n, **at)
    b = keep[0].cpu().numpy()
    q, s = b[16:16 + 2 * n * K].reshape(2, -1), b[at["s_off"]:at["s_off"] + 24].reshape(2, -1)
    blob = _dev(np.concatenate([s[1], s[0], np.zeros(8, np.uint8), q[1], q[0]]))
    t = torch.tensor([blob.data_ptr()], device="cuda")
    got = coli.fp8_swiglu(a, a_s, t, n, q_off=32 + n * K, s_off=12, up_q_off=32, up_s_off=0)
    assert torch.equal(got, want)


def test_not_finite(coli):
    """NaN codes and scales reach the results that they belong to and no other, in tails too."""
    import torch
    rng = np.random.default_rng(9)
    for K in (144, 512):
        a, a_s, _ = _rows(rng, 40, K)
        keep, table, _, at = _weights(rng, 1, 33, K)
        a[3, K - 1] = 0x7F
        a_s[5, -1] = float("nan")
        keep[0, 16 + 7 * K] = 0xFF
        for dtype in DTYPES:
            y = coli.fp8_matmul(a, a_s, table, 33, dtype=_t(dtype), **at).isnan()
            want = torch.zeros(40, 33, dtype=torch.bool, device="cuda")
            want[3], want[5], want[:, 7] = True, True, True
            assert torch.equal(y, want)


def test_offsets_that_c_would_cut(coli):
    """Byte offsets and truth values of more bits than the C types have."""
    import torch
    rng = np.random.default_rng(10)
    a, a_s, _ = _rows(rng, 3, 144)
    _keep, table, _, at = _weights(rng, 1, 32, 144, parts=2)
    for how in (dict(q_off=2 ** 64 + 16), dict(s_off=2 ** 64 + at["s_off"]), dict(q_off=-16), dict(s_off=-4)):
        for call in (coli.fp8_matmul, coli.fp8_swiglu):
            with pytest.raises(ValueError, match="2\\^63"):
                call(a, a_s, table, 32, **{**at, **how})
    for how in (dict(up_q_off=2 ** 64), dict(up_s_off=2 ** 64), dict(up_q_off=-16)):
        with pytest.raises(ValueError, match="2\\^63"):
            coli.fp8_swiglu(a, a_s, table, 32, **at, **how)
    gt, gs = coli.quantize_fp8_columns(torch.ones(5, 16, device="cuda"))
    out = torch.ones(1, 16, 16, device="cuda")
    assert bool((coli.fp8_wgrad(gt, gs, gt, gs, out=out, accumulate=2 ** 32) == 6.0).all())
    l = torch.randn(3, 8, device="cuda")
    assert torch.equal(coli.route_groups(l, None, 2, norm=2 ** 32)[1], coli.route_groups(l, None, 2)[1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,K,n", [(40, 144, 33), (40, 512, 33), (5, 640, 4100), (40, 656, 161), (9000, 16, 1300), (700, 640, 1500),
                                      (4500, 1152, 2060), (64, 8208, 8192)])
def test_infinite_scales(coli, rows, K, n, dtype):
    """An infinite scale of the last block, of a row and of the matrix, gives infinities of the products' signs (codes above 0 on
    both sides, one row's below) and nothing else, SwiGLU's too."""
    import torch
    rng = np.random.default_rng(rows + K)
    q, blocks = _codes(rng, n, K) & 0x7F, -(-K // 128)
    s = _scales(rng, 2e-3, -(-n // 128), blocks)
    s[-1, -1] = float("inf")                                      # of the last matrix rows
    at = (n - 1) // 128 * 128
    size = -(-(n * K + 4 * s.numel()) // 16) * 16
    blob = torch.zeros(2 * size, dtype=torch.uint8, device="cuda")
    blob[:n * K] = q.flatten()
    blob[n * K:n * K + 4 * s.numel()] = s.flatten().view(torch.uint8)
    blob[size:size + n * K] = q.flatten()                          # up: the same with finite scales
    blob[size + n * K:size + n * K + 4 * s.numel()] = s.nan_to_num(posinf=1e-3).flatten().view(torch.uint8)
    table = torch.tensor([blob.data_ptr()], device="cuda")
    a, a_s, _ = _rows(rng, rows, K, 1e-4)
    a &= 0x7F
    want = torch.zeros(rows, n, dtype=torch.bool, device="cuda")
    want[:, at:] = True
    y = coli.fp8_matmul(a, a_s, table, n, s_off=n * K, dtype=_t(dtype))
    assert not bool(y.isnan().any()) and torch.equal(y.isinf(), want) and bool((y > 0).all())
    h = coli.fp8_swiglu(a, a_s, table, n, s_off=n * K, up_q_off=size, up_s_off=size + n * K, dtype=_t(dtype))
    assert not bool(h.isnan().any()) and torch.equal(h.isinf(), want)
    a_s[1, -1] = float("inf")
    a[1] |= 0x80
    want[1] = True
    y = coli.fp8_matmul(a, a_s, table, n, s_off=n * K, dtype=_t(dtype))
    assert not bool(y.isnan().any()) and torch.equal(y.isinf(), want)
    assert bool((y[1] < 0).all()) and bool((y[torch.arange(rows, device="cuda") != 1] > 0).all())


@pytest.mark.parametrize("odd", (0, 4))
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,K,n,before,behind", [(150, 5136, 4100, 0, 0), ([130, 0, 123], 8192, 1030, 3, 4),
                                                      (64, 8192, 8192, 0, 0), ([1, 257, 0, 40], 8208, 777, 0, 2)],
                         ids=lambda v: str(v).replace(" ", ""))
def test_matmul_parts(coli, counts, K, n, before, behind, dtype, odd):
    """Columns summed in parts, in a workspace: another order of the same sums; rows outside the offsets stay."""
    import torch
    offsets, off, rows = _groups(counts, before, behind)
    E, exact = len(off) - 1, dtype == "float32"
    assert coli._fp8_matmul_ws(rows, K, E, n, offsets is not None, 1) > 0 or n == 777
    rng = np.random.default_rng(K + n + 2)
    _keep, table, matrix, at = _weights(rng, E, n, K, odd=odd)
    a, a_s, va = _rows(rng, rows, K)
    y, terms = _product(va, matrix, off, n)
    out = torch.full((rows, n + 3), 7.0, dtype=_t(dtype), device="cuda")
    coli.fp8_matmul(a, a_s, table, n, offsets=offsets, out=out[:, :n], **at)
    lo, hi = int(off[0]), int(off[-1])
    assert bool((out[:, n:] == 7.0).all()) and bool((out[:lo] == 7.0).all()) and bool((out[hi:] == 7.0).all())
    err, y = (out[lo:hi, :n].double() - y[lo:hi]).abs(), y[lo:hi]
    assert bool((err <= ref.product_bound(K, terms[lo:hi], exact) * (1 + _half_step(dtype)) + _half(dtype, y)).all())
    assert float(err.norm()) <= (ref.norm_bound(K, exact) + _half_step(dtype)) * float(y.norm())
    again = coli.fp8_matmul(a, a_s, table, n, offsets=offsets, dtype=_t(dtype), **at)
    assert torch.equal(again[lo:hi], out[lo:hi, :n])
    a[lo + 1, K - 1] = 0x7F                                       # a NaN in one part
    bad = coli.fp8_matmul(a, a_s, table, n, offsets=offsets, dtype=_t(dtype), **at)[lo:hi].isnan()
    assert bool(bad[1].all()) and int(bad.sum()) == n


def test_products_past_32_bits(coli):
    """Rows, matrices and outputs that lie beyond 2^32 bytes or 2^31 values: codes 1, scales 1 and 2, so that sums are whole."""
    import torch
    one = 0x38
    rows, n = 40000, 65552                                        # 2.6e9 outputs
    a = torch.full((rows, 16), one, dtype=torch.uint8, device="cuda")
    a_s = torch.ones(rows, 1, device="cuda")
    a_s[-1] = 2.0
    blob = torch.full((n * 16 + 4 * 513,), one, dtype=torch.uint8, device="cuda")
    blob[n * 16:] = torch.ones(513, device="cuda").view(torch.uint8)
    table = torch.tensor([blob.data_ptr()], device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        y = coli.fp8_matmul(a, a_s, table, n, s_off=n * 16, dtype=dtype)
        assert y.max().item() == 32.0 and bool((y[-1] == 32.0).all()) and bool((y[:-1:997] == 16.0).all()) and y[-2].min().item() == 16.0
        del y
    rows, K, n = 70000, 65536, 144                                # 4.6e9 codes of rows
    a = torch.zeros(rows, K, dtype=torch.uint8, device="cuda")
    a[-1], a[-2, -1] = one, one
    a_s = torch.ones(rows, 512, device="cuda")
    w = torch.full((n * K + 4 * 1024,), one, dtype=torch.uint8, device="cuda")
    w[n * K:] = torch.ones(1024, device="cuda").view(torch.uint8)
    table = torch.tensor([w.data_ptr()], device="cuda")
    off = torch.tensor([0, rows - 3, rows], dtype=torch.int32, device="cuda")
    for kw in (dict(), dict(offsets=off)):
        y = coli.fp8_matmul(a, a_s, table.repeat(2) if kw else table, n, s_off=n * K, dtype=torch.bfloat16, **kw)
        assert bool((y[-1] == 65536.0).all()) and bool((y[-2] == 1.0).all()) and bool((y[:-2] == 0).all())
    del a, y
    n = (1 << 29) + 16                                            # more matrix rows than few_rows' launches take
    w = torch.full((16 * n + 4 * (n // 128 + 1),), one, dtype=torch.uint8, device="cuda")
    w[16 * n:].view(torch.float32).fill_(0.5)
    w[16 * (n - 1):16 * n] = 0x40
    for dtype in (torch.bfloat16, torch.float32):
        y = coli.fp8_matmul(torch.full((1, 16), one, dtype=torch.uint8, device="cuda"), torch.ones(1, 1, device="cuda"),
                            torch.tensor([w.data_ptr()], device="cuda"), n, s_off=16 * n, dtype=dtype)
        assert y[0, -1].item() == 16.0 and bool((y[0, :-1] == 8.0).all())
    del w, y
    n = 70000                                                     # 4.6e9 codes of a matrix, and one row
    w = torch.zeros(n * K + 4 * 547 * 512, dtype=torch.uint8, device="cuda")
    w[(n - 1) * K:n * K] = one
    w[n * K:].view(torch.float32).fill_(2.0)
    table = torch.tensor([w.data_ptr()], device="cuda")
    for rows in (1, 300):
        a, a_s = torch.full((rows, K), one, dtype=torch.uint8, device="cuda"), torch.ones(rows, 512, device="cuda")
        y = coli.fp8_matmul(a, a_s, table, n, s_off=n * K)
        assert bool((y[:, -1] == 131072.0).all()) and bool((y[:, :-1] == 0).all())


def test_wgrad_past_32_bits(coli):
    import torch
    E, n, K = 3, 30016, 30000                                     # 2.7e9 gradients
    g, x = torch.zeros(4, n, device="cuda"), torch.ones(4, K, device="cuda")
    g[-1, -1] = 2.0
    off = torch.tensor([0, 1, 1, 4], dtype=torch.int32, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        dw = coli.fp8_wgrad(*coli.quantize_fp8_columns(g, off), *coli.quantize_fp8_columns(x, off), off, dtype=dtype)
        assert bool((dw[2, -1] == 2.0).all()) and bool((dw[2, :-1] == 0).all()) and bool((dw[:2] == 0).all())
        del dw
    rows, n, K = 40000, 65552, 16                                 # 2.6e9 codes of columns, 16-bit: 2^32 bytes of values
    g, x = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda"), torch.ones(rows, K, device="cuda")
    g[-1, -1], g[0, 0] = 2.0, 3.0
    dw = coli.fp8_wgrad(*coli.quantize_fp8_columns(g), *coli.quantize_fp8_columns(x), rows=rows)
    assert bool((dw[0, -1] == 2.0).all()) and bool((dw[0, 0] == 3.0).all()) and bool((dw[0, 1:-1] == 0).all())


# ---------------------------------------------------------------- gradients
WGRAD = [([3], 16, 16), ([128, 0, 129, 1], 144, 272), ([5, 40, 0, 260, 17], 64, 528), ([0, 0], 32, 16), ([1] * 9, 128, 128), (300, 272, 144),
         ([700], 528, 400), ([5, 0, 130], 1168, 272), ([40, 3], 144, 1024), (1400, 48, 80),
         ([6000, 0, 1500, 20], 48, 272), ([3, 8100], 272, 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,n,K", WGRAD, ids=lambda v: str(v).replace(" ", ""))
def test_wgrad(coli, counts, n, K, dtype):
    import torch
    before, behind = (0, 0) if isinstance(counts, int) else (2, 3)
    offsets, off, rows = _groups(counts, before, behind)
    E = len(off) - 1
    rng = np.random.default_rng(n + K)
    g, x = 0.05 * rng.standard_normal((rows, n)), rng.standard_normal((rows, K)) * np.exp2(rng.integers(-6, 6, K))
    g, x = _dev(g).to(torch.bfloat16), _dev(x).to(torch.bfloat16)
    cols = [(coli.quantize_fp8_columns(t, offsets)) for t in (g, x)]
    want, terms = np.zeros((E, n, K)), np.zeros((E, n, K))
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        vals = []
        for t in (g, x):
            q, s = ref.quantize_columns(_host(t)[lo:hi], [0, hi - lo])
            vals.append(ref.column_values(q, s))
        want[e], terms[e] = vals[0] @ vals[1].T, np.abs(vals[0]) @ np.abs(vals[1]).T
    most = max(1, int((off[1:] - off[:-1]).max()))
    tol = ref.product_bound(most, terms, dtype == "float32")
    got = coli.fp8_wgrad(*cols[0], *cols[1], offsets, dtype=_t(dtype))
    assert got.shape == (E, n, K)
    err = np.abs(_host(got) - want)
    assert _within(err, tol * (1 + _half_step(dtype)) + _rounding(dtype, want))
    assert np.linalg.norm(err) <= (ref.norm_bound(most, dtype == "float32") + _half_step(dtype)) * np.linalg.norm(want)
    # added to what is there, into rows with a gap
    buf = torch.full((E, n, K + 3), 2.0, dtype=_t(dtype), device="cuda")
    coli.fp8_wgrad(*cols[0], *cols[1], offsets, out=buf[..., :K], accumulate=True)
    assert bool((buf[..., K:] == 2.0).all())
    err = np.abs(_host(buf[..., :K]) - want - 2.0)
    assert _within(err, tol * 1.01 + (_half_step(dtype) + 2.0 ** -24) * (np.abs(want) + 2.0))
    coli.fp8_wgrad(*cols[0], *cols[1], offsets, out=buf[..., :K])
    assert torch.equal(buf[..., :K], got)


@pytest.mark.parametrize("size", (1e-30, 1e-35, 1e-36, 1e-38, 1e-39))
def test_wgrad_of_the_smallest_scales(coli, size):
    """Gradients next to the smallest numbers: exact from a scale of 2^-124 on, below rounded to multiples of 2^-133 in f32
    results, half of that off at most, times the other operand; the FP8 instruction takes the scales as they are."""
    import torch
    rng = np.random.default_rng(15)
    rows, n, K = 300, 32, 144
    x = 1e8 * rng.standard_normal((rows, K))
    g = size * rng.standard_normal((rows, n))
    cols = [coli.quantize_fp8_columns(_dev(t.astype(np.float32))) for t in (g, x)]
    vals = [ref.column_values(q.cpu().numpy(), s.cpu().numpy().astype(np.int64)) for q, s in cols]
    want, terms = vals[0] @ vals[1].T, np.abs(vals[0]) @ np.abs(vals[1]).T
    code = cols[0][1].cpu().numpy()
    assert code.max() < 3 if size < 5e-36 else code.min() >= 3
    lost = 0.0 if size >= 5e-36 else 2.0 ** -134 * np.abs(vals[1]).sum(1)
    for dtype in ("float32", "bfloat16"):
        exact = dtype == "float32"
        got = _host(coli.fp8_wgrad(*cols[0], *cols[1], rows=rows, dtype=_t(dtype))[0])
        tol = ref.product_bound(rows, terms, exact) + (lost if exact else 0.0)
        assert (np.abs(got - want) <= tol * (1 + _half_step(dtype)) + _rounding(dtype, want)).all()


def test_wgrad_parts(coli):
    """Rows summed in parts (with a workspace) and at once (without) agree, NaN included, and repeat bit for bit. f32: about
    160 additions of 32 products each round by 2^-25 of sums that do not exceed the largest result by much, 13 * 2^-25 as
    independent errors on each side, and 2^5 to spare; bf16: one rounding on each side, 2^-8 each."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    for counts, n, K in (([2900, 1], 144, 272), (5000, 16, 1040)):
        offsets, off, rows = _groups(counts, 0, 0)
        E = len(off) - 1
        a, b = torch.randn(rows, n, device="cuda", generator=g), torch.randn(rows, K, device="cuda", generator=g)
        a[17, 3], b[rows - 1, 5] = float("nan"), float("inf")
        (ga, gs), (xa, xs) = coli.quantize_fp8_columns(a, offsets), coli.quantize_fp8_columns(b, offsets)
        assert coli._fp8_wgrad_ws(rows, E, n, K) > 0
        for dtype, code in ((torch.float32, 0), (torch.bfloat16, 1)):
            got = coli.fp8_wgrad(ga, gs, xa, xs, offsets, rows=rows, dtype=dtype)
            one = torch.empty_like(got)
            assert coli.lib().coli_fp8_wgrad(ga.data_ptr(), gs.data_ptr(), xa.data_ptr(), xs.data_ptr(), ga.shape[0], rows,
                                             None if offsets is None else offsets.data_ptr(), E, n, K, 0, one.data_ptr(), code, K,
                                             None, 0, coli._stream()) == 0
            assert torch.equal(got.isnan(), one.isnan()) and bool(got[0, 3].isnan().all())
            scale = float(one.nan_to_num(0.0).double().abs().max())
            assert float((got - one).nan_to_num(0.0).double().abs().max()) <= (2.0 ** -15 if code == 0 else 2.0 ** -7) * scale
            again = coli.fp8_wgrad(ga, gs, xa, xs, offsets, rows=rows, dtype=dtype)
            assert torch.equal(again.nan_to_num(7.0), got.nan_to_num(7.0))


def test_wgrad_not_finite_and_no_rows(coli):
    import torch
    off = _dev(np.array([0, 0, 5], np.int32))
    g, x = torch.ones(5, 16, device="cuda"), torch.ones(5, 32, device="cuda")
    g[2, 3], x[1, 7] = float("nan"), float("inf")
    for dtype in DTYPES:
        dw = coli.fp8_wgrad(*coli.quantize_fp8_columns(g, off), *coli.quantize_fp8_columns(x, off), off, dtype=_t(dtype))
        assert bool((dw[0] == 0).all())
        bad = torch.zeros(16, 32, dtype=torch.bool, device="cuda")
        bad[3], bad[:, 7] = True, True
        assert torch.equal(dw[1].isnan(), bad) and bool((dw[1][~bad] == 5.0).all())
        none = torch.zeros(3, dtype=torch.int32, device="cuda")
        cols = coli.quantize_fp8_columns(g[:0], none), coli.quantize_fp8_columns(x[:0], none)
        out = torch.full((2, 16, 32), 3.0, dtype=_t(dtype), device="cuda")
        coli.fp8_wgrad(*cols[0], *cols[1], none, out=out, accumulate=True)
        assert bool((out == 3.0).all())
        assert bool((coli.fp8_wgrad(*cols[0], *cols[1], none, out=out) == 0).all())


def test_layer_forward_and_backward(coli):
    """The operators as a training step runs them, against the same steps in 64 bits from the same choices and
    quantised values; the matrices' gradient also against differences."""
    import torch
    rng = np.random.default_rng(11)
    T, k, E, H, I = 70, 3, 8, 272, 144
    x = _dev(rng.standard_normal((T, H))).to(torch.bfloat16)
    logits, bias = _dev(rng.standard_normal((T, E)).astype(np.float32)), _dev(0.1 * rng.standard_normal(E).astype(np.float32))
    logits[4] = -float("inf")                                     # a padded token
    W = _dev(0.05 * rng.standard_normal((E, I, H))).to(torch.bfloat16)
    q, s, qt, st = coli.quantize_fp8_matrix(W, transposed=True)

    def table(q, s):
        n = q[0].numel()
        blobs = torch.zeros(E, -(-(n + 4 * s[0].numel()) // 16) * 16, dtype=torch.uint8, device="cuda")
        blobs[:, :n] = q.flatten(1)
        blobs[:, n:n + 4 * s[0].numel()] = s.flatten(1).contiguous().view(torch.uint8)
        return blobs, blobs.data_ptr() + blobs.shape[1] * torch.arange(E, device="cuda"), n

    keep, tab, s_off = table(q, s)
    keep_t, tab_t, s_off_t = table(qt, st)
    idx, w = coli.route_groups(logits, bias, k, groups=4, groups_kept=2, scale=2.0)
    _, offsets, _, _, _, inv = coli.union_inverse(idx, E)
    a, a_s = coli.dispatch_fp8(x, inv)
    rows = coli.fp8_matmul(a, a_s, tab, I, s_off=s_off, offsets=offsets)
    y = coli.combine(rows, inv, w)
    dy = _dev(rng.standard_normal((T, I)).astype(np.float32))
    d_rows, d_w = coli.combine_bwd(dy, rows, inv, w)
    gt, gt_s, g, g_s = coli.quantize_fp8_columns(d_rows, offsets, rows=True)
    d_a = coli.fp8_matmul(g, g_s, tab_t, H, s_off=s_off_t, offsets=offsets)
    xr = coli.dispatch(x, inv)
    dW = coli.fp8_wgrad(gt, gt_s, *coli.quantize_fp8_columns(xr, offsets), offsets)
    dx = coli.dispatch_bwd(d_a, inv)
    dl = coli.route_groups_bwd(d_w, logits, idx, scale=2.0)
    # the same in 64 bits
    vx = ref.values(*[f(t) for f, t in zip((lambda t: t, ref.scale_value), ref.quantize_rows(_host(x)))])
    vW = _host(coli.dequantize_fp8(q, s))
    ii, ww = idx.cpu().numpy(), _host(w)
    off, place = offsets.cpu().numpy(), inv.cpu().numpy()
    assert (place[4] == -1).all() and int(off[-1]) == (T - 1) * k and (ii[4] == -1).all()
    yr, drows = np.zeros((T, I)), np.zeros((T * k, I))
    dwr, xrow = np.zeros((T, k)), np.zeros((T * k, H))
    for t in range(T):
        for j in range(k):
            if ii[t, j] >= 0:
                r = vW[ii[t, j]] @ vx[t]
                yr[t] += ww[t, j] * r
                dwr[t, j] = _host(dy)[t] @ r
                drows[place[t, j]] = ww[t, j] * _host(dy)[t]
                xrow[place[t, j]] = _host(x)[t]
    assert np.linalg.norm(_host(y) - yr) <= 1e-5 * np.linalg.norm(yr)
    assert np.linalg.norm(_host(d_w) - dwr) <= 1e-5 * np.linalg.norm(dwr)
    assert np.linalg.norm(_host(dl) - ref.route_grad(dwr, _host(logits), ii, "sigmoid", True, 2.0)) <= 1e-4 * np.linalg.norm(_host(dl))
    assert bool((dl[4] == 0).all()) and bool((dx[4] == 0).all())
    used = int(off[-1])
    dr = _host(d_rows)[:used]                                     # the quantisers' own inputs
    qg, sg = ref.quantize_rows(dr)
    vg, da = ref.values(qg, ref.scale_value(sg)), np.zeros((T * k, H))
    for e in range(E):
        da[off[e]:off[e + 1]] = vg[off[e]:off[e + 1]] @ vW[e]
    dxr = np.stack([sum((da[p] for p in place[t] if p >= 0), np.zeros(H)) for t in range(T)])
    assert np.linalg.norm(_host(dx) - dxr) <= 1e-5 * np.linalg.norm(dxr)
    vals = []
    for t in (dr, xrow[:used]):
        qc, sc = ref.quantize_columns(t, off)
        vals.append(ref.column_values(qc, sc))
    first = np.concatenate([[0], np.cumsum(-(-(off[1:] - off[:-1]) // 128) * 128)])
    for e in range(E):
        gv, xv = vals[0][:, first[e]:first[e + 1]], vals[1][:, first[e]:first[e + 1]]
        assert np.linalg.norm(_host(dW[e]) - gv @ xv.T) <= 1e-5 * np.linalg.norm(gv @ xv.T)
        D = rng.standard_normal((I, H))                           # f(W) = sum of g . W x is linear: its difference is <dW, D>
        diff = ((gv * ((vW[e] + D) @ xv)).sum() - (gv * ((vW[e] - D) @ xv)).sum()) / 2
        assert abs((_host(dW[e]) * D).sum() - diff) <= 1e-4 * np.linalg.norm(gv @ xv.T) * np.linalg.norm(D) / np.sqrt(D.size) * 40


def test_graph_and_streams(coli):
    """A layer, forward and backward, in a graph that is replayed with new inputs, and on a given stream."""
    import torch
    rng = np.random.default_rng(12)
    K, n, E, rows = 640, 256, 3, 30
    keep, table, _, at = _weights(rng, E, n, K, parts=2)
    off = _dev(np.array([0, 9, 9, 30], np.int32))
    x = torch.randn(rows, K, device="cuda").to(torch.bfloat16)
    keep2, table2, _, at2 = _weights(rng, E, K, n)
    B = coli.fp8_column_blocks(rows, E)
    e = torch.empty
    out = dict(q=e(rows, K, dtype=torch.uint8, device="cuda"), s=e(rows, 5, device="cuda"), h=e(rows, n, dtype=torch.uint8, device="cuda"),
               hs=e(rows, 2, device="cuda"), y=e(rows, K, device="cuda"), qt=e(B, K, 128, dtype=torch.uint8, device="cuda"),
               st=e(B, K, dtype=torch.uint8, device="cuda"), dw=e(E, K, K, device="cuda"), v=e(rows, K, device="cuda"))

    def step(o, stream=None):
        coli.quantize_fp8_columns(x, off, qt=o["qt"], st=o["st"], q=o["q"], s=o["s"], stream=stream)
        coli.fp8_swiglu(o["q"], o["s"], table, n, offsets=off, out=(o["h"], o["hs"]), stream=stream, **at)
        coli.fp8_matmul(o["h"], o["hs"], table2, K, offsets=off, out=o["y"], stream=stream, **at2)
        coli.fp8_wgrad(o["qt"], o["st"], o["qt"], o["st"], off, out=o["dw"], stream=stream)
        coli.dequantize_fp8(o["q"], o["s"], out=o["v"], stream=stream)

    step(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    side = torch.cuda.Stream()
    for seed in range(3):
        x.copy_(torch.randn(rows, K, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        other = {k: torch.zeros_like(v) for k, v in out.items()}
        side.wait_stream(torch.cuda.current_stream())
        step(other, side)
        side.synchronize()
        assert torch.equal(out["y"], other["y"]) and torch.equal(out["dw"], other["dw"]) and torch.equal(out["v"], other["v"])
        assert torch.equal(out["h"], other["h"])


def test_two_graphs_at_once(coli):
    """Two captured layers of few rows, whose SwiGLU takes a workspace, replayed at the same time on two streams."""
    import torch
    rng = np.random.default_rng(13)
    K, n, E, rows = 2048, 640, 4, 4
    off = _dev(np.array([0, 1, 1, 3, 4], np.int32))
    runs = []
    for i in range(2):
        keep, table, _, at = _weights(rng, E, n, K, parts=2, odd=0)
        x = torch.randn(rows, K, device="cuda")
        graph = torch.cuda.CUDAGraph()

        def layer(x=x, table=table, at=at):
            q, s = coli.quantize_fp8(x)
            return coli.fp8_swiglu(q, s, table, n, offsets=off, dtype="fp8", **at)

        layer()
        with torch.cuda.graph(graph):
            out = layer()
        runs.append((keep, layer, x, graph, out, torch.cuda.Stream()))
    assert coli.debug_fp8_kernel(rows, K, E, n, grouped=True, swiglu=True) == "few_rows_32"
    for seed in range(4):
        for i, (_, _, x, _, _, stream) in enumerate(runs):
            x.copy_(torch.randn(rows, K, generator=torch.Generator().manual_seed(2 * seed + i)))
            stream.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            for _, _, _, graph, _, stream in runs:
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for _, layer, _, _, out, _ in runs:
            want = layer()
            assert torch.equal(want[0], out[0]) and torch.equal(want[1], out[1])


def test_parts_in_graphs(coli):
    """Products and gradients in parts, in two graphs with workspaces of their own, replayed at the same time."""
    import torch
    rng = np.random.default_rng(14)
    rows, K, n = 150, 5136, 4100
    assert coli._fp8_matmul_ws(rows, K, 1, n, False, 1) > 0 and coli._fp8_wgrad_ws(3000, 1, 48, 80) > 0
    runs = []
    for _ in range(2):
        keep, table, _, at = _weights(rng, 1, n, K, odd=0)
        x, g, y = (torch.randn(*s, device="cuda") for s in ((rows, K), (3000, 48), (3000, 80)))

        def step(x=x, g=g, y=y, table=table, at=at):
            out = coli.fp8_matmul(*coli.quantize_fp8(x), table, n, dtype=torch.bfloat16, **at)
            return out, coli.fp8_wgrad(*coli.quantize_fp8_columns(g), *coli.quantize_fp8_columns(y), rows=3000)

        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        runs.append((keep, step, (x, g, y), graph, out, torch.cuda.Stream()))
    for seed in range(3):
        for i, (_, _, inputs, _, _, stream) in enumerate(runs):
            for t in inputs:
                t.copy_(torch.randn(*t.shape, generator=torch.Generator().manual_seed(2 * seed + i)))
            stream.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            for _, _, _, graph, _, stream in runs:
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for _, step, _, _, out, _ in runs:
            want = step()
            assert torch.equal(want[0], out[0]) and torch.equal(want[1], out[1])
