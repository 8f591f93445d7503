"""MXFP4 quantiser and grouped products against plain 64-bit forms.

Tolerances: the quantiser and its inverse are exact. Products: product_bound's
argument for the f32 sums, plus half a step of the output type. SwiGLU: the
errors of both sums through the derivatives (|silu'| <= 1.1), 16 half-steps of
f32 for exp, divide and the two products, plus the output's half step."""
import numpy as np
import pytest

from tests import mxfp4_refs as ref

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


def _host(t):
    return t.double().cpu().numpy()


def _hard_rows(rng, rows, cols, scale=1.0):
    """Normal values with ties, exact binade ends, zeros, outliers and wide ranges among them."""
    x = rng.standard_normal((rows, cols)) * scale
    x *= np.exp2(rng.integers(-8, 9, (rows, cols // 32))).repeat(32, 1)
    x = x.reshape(rows, -1, 32)
    x[rng.random(x.shape[:2]) < 0.1] = 0.0
    ties = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], x.shape) * rng.choice([-1, 1], x.shape)
    pick = rng.random(x.shape[:2]) < 0.3
    x[pick] = (ties * np.exp2(rng.integers(-6, 6, x.shape[:2]))[..., None])[pick]
    x[rng.random(x.shape) < 0.02] = -0.0
    return x.reshape(rows, cols)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (3, 96, 0), (1, 6144, 0), (37, 2080, 0), (37, 2080, 5),
                                           (1029, 1056, 0), (513, 2048, 8)])
def test_quantize_matches_reference(coli, dtype, rows, cols, pad):
    import torch
    rng = np.random.default_rng(rows * 1000 + cols + pad)
    full = torch.from_numpy(_hard_rows(rng, rows, cols)).to(_t(dtype))
    buf = torch.full((rows, cols + pad), float("nan"), dtype=_t(dtype))
    buf[:, :cols] = full
    x = buf.to("cuda")[:, :cols]
    q, s = coli.quantize_mxfp4(x)
    qr, sr = ref.quantize(_host(full))
    assert np.array_equal(s.cpu().numpy(), sr)
    assert np.array_equal(q.cpu().numpy(), qr)
    for out in DTYPES:
        out_buf = torch.full((rows, cols + pad), 7.0, dtype=_t(out), device="cuda")
        v = coli.dequantize_mxfp4(q, s, out=out_buf[:, :cols])
        want = torch.from_numpy(ref.values(qr, sr)).to(_t(out))
        assert torch.equal(v.cpu(), want)
        assert bool((out_buf[:, cols:] == 7.0).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_extremes(coli, dtype):
    """Infinities, NaN, the type's largest and smallest values, empty input; rows off a
    16-byte boundary."""
    import torch
    info = torch.finfo(_t(dtype))
    x = torch.zeros(8, 64, dtype=_t(dtype))
    x[0, 3] = float("inf")
    x[0, 33] = float("-inf")
    x[1, 31], x[1, 40] = float("nan"), 1.0
    x[2] = info.max
    x[3] = info.min
    x[4] = info.tiny
    x[5, :32] = info.smallest_normal * info.eps               # subnormal
    x[6, 0], x[6, 1] = info.max, info.tiny
    x[7, 0] = info.tiny / 4
    q, s = coli.quantize_mxfp4(x.to("cuda"))
    qr, sr = ref.quantize(_host(x))
    assert np.array_equal(s.cpu().numpy(), sr) and np.array_equal(q.cpu().numpy(), qr)
    assert sr[0].tolist() == [255, 255] and sr[1, 0] == 255 and sr[1, 1] != 255
    v = coli.dequantize_mxfp4(q, s)
    assert np.array_equal(_host(v), ref.values(qr, sr), equal_nan=True)
    for out in ("float16", "bfloat16"):                       # beyond float16's range: infinity
        want = torch.from_numpy(ref.values(qr, sr)).to(_t(out))
        assert torch.equal(coli.dequantize_mxfp4(q, s, dtype=_t(out)).cpu().nan_to_num(9.0), want.nan_to_num(9.0))
    buf = torch.zeros(8 * 64 + 1, dtype=_t(dtype), device="cuda")
    odd = buf[1:].view(8, 64)
    odd.copy_(x)
    q2, s2 = coli.quantize_mxfp4(odd)
    assert torch.equal(q2, q) and torch.equal(s2, s)
    q0, s0 = coli.quantize_mxfp4(torch.empty(0, 64, dtype=_t(dtype), device="cuda"))
    assert q0.shape == (0, 32) and s0.shape == (0, 2)
    assert coli.dequantize_mxfp4(q0, s0).shape == (0, 64)


def test_quantize_past_32_bits(coli):
    """More than 2^32 bytes and 2^31 values in, a far block written where it belongs."""
    import torch
    rows, cols = 1 << 18, 8224                                  # 2.16e9 bf16 values
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1, -32:] = 3.0
    x[rows // 2, 32] = -1.0
    for src in (x, x[:, :8192]):                                # gapless, then strided rows
        q, s = coli.quantize_mxfp4(src)
        assert q[rows // 2, 16].item() == 0xE and s[rows // 2, 1].item() == 125
        assert int(s.long().sum()) == 125 + (126 if src is x else 0)
        if src is x:
            assert s[-1, -1].item() == 126 and (q[-1, -16:] == 0x77).all()
            v = coli.dequantize_mxfp4(q, s, dtype=torch.bfloat16)
            assert (v[-1, -32:] == 3.0).all() and v[rows // 2, 32].item() == -1.0
            assert int((v != 0).sum()) == 33
            del v
        del q, s


class Mats:
    """E random MXFP4 matrices as device buffers (codes, then scales at an offset of 5 past 16 bytes, or
    aligned to them) and in 64 bits."""

    def __init__(self, coli, rng, E, N, K, lo=117, hi=130, aligned=False):
        self.q_off, self.s_off = 32, 32 + N * K // 2 + (0 if aligned else 5)
        self.values, blobs = [], []
        for e in range(E):
            q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
            s = rng.integers(lo, hi, (N, K // 32), dtype=np.uint8)
            blob = np.zeros(self.s_off + N * K // 32, np.uint8)
            blob[self.q_off:self.q_off + N * K // 2] = q.ravel()
            blob[self.s_off:] = s.ravel()
            blobs.append(_dev(blob))
            self.values.append(ref.values(q, s))
        self.blobs = blobs
        self.table = coli.blob_table(blobs)


def _rows(rng, R, K, lo=117, hi=130):
    q = rng.integers(0, 256, (R, K // 2), dtype=np.uint8)
    s = rng.integers(lo, hi, (R, K // 32), dtype=np.uint8)
    return q, s, ref.values(q, s)


def _counts_to_offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


# counts per expert (None: one matrix without offsets, R rows), N, K, spare rows behind the last
CASES = [
    ([1], 16, 32, 0), ([0, 1, 0], 17, 64, 0), ([3, 0, 2], 5, 96, 2), (1, 1, 32, 0), (5, 33, 160, 0),
    ([1, 1, 0, 1], 64, 512, 0), ([16, 17, 0, 15, 1], 100, 544, 3), ([40, 0, 7], 130, 1120, 1),
    (61, 257, 2048, 0), ([64, 65, 63, 0, 128, 1], 272, 640, 9), ([200, 3], 96, 1056, 0), (300, 300, 480, 0),
    ([0, 0, 0], 64, 128, 4), ([129] + [0] * 70 + [3] + [0] * 200 + [31], 48, 256, 0), (257, 129, 4640, 0),
]


def _case(coli, rng, counts, N, K, spare, aligned=False, **kw):
    if isinstance(counts, int):
        off, R, E = None, counts, 1
        off_np = np.array([0, counts])
    else:
        off_np = _counts_to_offsets(counts)
        R, E = int(off_np[-1]) + spare, len(counts)
        off = _dev(off_np)
    mats = Mats(coli, rng, E, N, K, aligned=aligned, **kw)
    q, s, a = _rows(rng, R, K, **kw)
    if spare:                                                   # rows of no expert hold NaN
        s[-spare:] = 255
    return mats, _dev(q), _dev(s), a, off, off_np, R


# the same with scales on 16-byte boundaries and columns in 512s: rows per expert around the tiles of 128 and 256,
# empty experts between them, more units than workgroups, one unit, matrix rows that end inside a tile
LINES = [([3], 256, 1024, 0), ([5, 0, 4, 130, 128, 129, 0], 300, 1024, 2), ([0] * 9 + [200], 77, 1536, 1),
         ([31, 33, 17, 16, 64, 65], 1000, 2048, 0), (257, 1030, 1024, 0), ([9] * 70, 1100, 1024, 5),
         ([1025, 1030], 4100, 1024, 3), (2300, 8300, 1024, 0), ([300] + [0] * 1022 + [7], 520, 1024, 0),
         ([0] * 300, 300, 1024, 700), ([0, 700] * 20, 1100, 1024, 0), ([2] * 500, 260, 1024, 0), ([3] * 500, 260, 1536, 0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,N,K,spare,aligned", [c + (False,) for c in CASES] + [c + (True,) for c in LINES])
def test_matmul_matches_reference(coli, dtype, counts, N, K, spare, aligned):
    import torch
    rng = np.random.default_rng(N * 7919 + K)
    mats, q, s, a, off, off_np, R = _case(coli, rng, counts, N, K, spare, aligned=aligned)
    pad = 3
    buf = torch.full((R, N + pad), 7.0, dtype=_t(dtype), device="cuda")
    y = coli.mxfp4_matmul(q, s, mats.table, N, mats.q_off, mats.s_off, offsets=off, out=buf[:, :N])
    want, terms = ref.product(a, mats.values, off_np)
    n = int(off_np[-1])
    got = _host(y)[:n]
    big = np.abs(want) > float(torch.finfo(_t(dtype)).max)
    assert not big.any()
    bound = ref.product_bound(K, terms[:n]) + _half_step(dtype) * (np.abs(want[:n]) + ref.product_bound(K, terms[:n]))
    bound += 2.0 ** -25 if dtype == "float16" else 0.0          # half a step below its normal range
    assert (np.abs(got - want[:n]) <= bound).all(), float((np.abs(got - want[:n]) / bound).max())
    assert bool((buf[:, N:] == 7.0).all()) and bool((buf[n:] == 7.0).all())


@pytest.mark.parametrize("R,N,K", [(1, 64, 2048), (16, 48, 6144), (70, 256, 1024), (260, 256, 2048), (130, 500, 2080),
                                   (300, 300, 5152), (1100, 520, 1536), (2100, 8200, 1024), (9, 40, 1056),
                                   (5, 70, 5152), (3, 33, 4096), (700, 520, 32), (300, 300, 96), (400, 260, 224),
                                   (500, 600, 480)])
def test_matmul_is_exact_where_f32_is(coli, R, N, K):
    """With scales within three binades on each side every partial sum has at most 24 bits."""
    rng = np.random.default_rng(R)
    for aligned in (False, True):
        mats = Mats(coli, rng, 1, N, K, 119, 121, aligned)
        q, s, a = _rows(rng, R, K, 126, 128)
        y = coli.mxfp4_matmul(_dev(q), _dev(s), mats.table, N, mats.q_off, mats.s_off)
        assert np.array_equal(_host(y), ref.product(a, mats.values, np.array([0, R]))[0])


def test_product_special_scales(coli):
    """NaN scales reach exactly the outputs that read them; the smallest and largest scales multiply."""
    import torch
    rng = np.random.default_rng(5)
    N, K, R = 40, 288, 21
    q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    s = np.full((N, K // 32), 127, np.uint8)
    s[7, 4], s[9, 8] = 255, 255
    aq = rng.integers(0, 256, (R, K // 2), dtype=np.uint8)
    as_ = np.full((R, K // 32), 127, np.uint8)
    as_[20, 8] = 255
    blob = _dev(np.concatenate([q.ravel(), s.ravel()]))
    y = _host(coli.mxfp4_matmul(_dev(aq), _dev(as_), coli.blob_table([blob]), N, 0, N * K // 2))
    bad = np.isnan(y)
    want = np.zeros((R, N), bool)
    want[:, [7, 9]] = True
    want[20] = True
    assert np.array_equal(bad, want)
    s[:], as_[:] = 0, 252                                       # 2^-127 and 2^125
    blob = _dev(np.concatenate([q.ravel(), s.ravel()]))
    y = coli.mxfp4_matmul(_dev(aq), _dev(as_), coli.blob_table([blob]), N, 0, N * K // 2)
    want = ref.values(aq, as_) @ ref.values(q, s).T             # at most 12 bits: exact
    assert np.array_equal(_host(y), want)


def _swiglu_ref(a, mats, off_np, K):
    want, terms = ref.product(a, mats.values, off_np)
    e = ref.product_bound(K, terms)
    pick = lambda z: [z.reshape(z.shape[0], -1, 2, 16)[:, :, i].reshape(z.shape[0], -1) for i in (0, 1)]
    (g, u), (eg, eu) = pick(want), pick(e)
    with np.errstate(over="ignore"):
        sg = g / (1 + np.exp(-g))
    h = sg * u
    bound = 1.1 * eg * (np.abs(u) + eu) + np.abs(sg) * eu + 16 * 2.0 ** -24 * np.abs(h) + 1e-37
    return h, bound


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,I,K,spare", [
    ([1], 32, 32, 0), ([0, 1, 2], 64, 96, 1), (5, 32, 544, 0), ([16, 17, 0, 1], 96, 640, 2),
    ([64, 1, 70], 160, 512, 0), (130, 288, 1056, 0), ([1] * 9, 256, 2048, 0), (260, 128, 256, 0),
    ([5, 0, 4, 130, 128, 129], 160, 1024, 2), ([40] * 40, 1056, 1024, 0), (2300, 4128, 1024, 0)])
@pytest.mark.parametrize("aligned", [False, True])
def test_swiglu_matches_reference(coli, dtype, counts, I, K, spare, aligned):
    import torch
    rng = np.random.default_rng(I + K)
    mats, q, s, a, off, off_np, R = _case(coli, rng, counts, 2 * I, K, spare, aligned=aligned, lo=120, hi=126)
    buf = torch.full((R, I + 1), 7.0, dtype=_t(dtype), device="cuda")
    h = coli.mxfp4_swiglu(q, s, mats.table, I, mats.q_off, mats.s_off, offsets=off, out=buf[:, :I])
    want, bound = _swiglu_ref(a, mats, off_np, K)
    n = int(off_np[-1])
    bound = bound[:n] + _half_step(dtype) * (np.abs(want[:n]) + bound[:n]) + (2.0 ** -25 if dtype == "float16" else 0)
    err = np.abs(_host(h)[:n] - want[:n])
    assert (err <= bound).all(), float((err / bound).max())
    assert bool((buf[:, I:] == 7.0).all()) and bool((buf[n:] == 7.0).all())


@pytest.mark.parametrize("counts,I,K,spare", [
    ([1], 32, 32, 0), ([0, 1, 2], 64, 96, 1), ([16, 17, 0, 1], 96, 640, 2), ([64, 1, 70], 160, 512, 0),
    (130, 288, 1024, 0), ([1] * 9, 256, 2048, 0), (300, 64, 512, 0), ([5, 0, 4, 130, 128, 129], 160, 1024, 2),
    ([40] * 40, 1056, 1024, 0), (2300, 4128, 1024, 0), ([150, 33], 96, 1056, 0), ([1, 0, 3], 64, 4640, 0),
    ([2, 1], 64, 4096, 1), ([700, 0, 9], 288, 96, 1), ([300, 600], 512, 224, 0)])
@pytest.mark.parametrize("aligned", [False, True])
def test_swiglu_to_mxfp4(coli, counts, I, K, spare, aligned):
    """The quantised output is the quantiser's answer to the f32 output (sums exact by the choice of scales)."""
    import torch
    rng = np.random.default_rng(I * 3 + K)
    mats, q, s, a, off, off_np, R = _case(coli, rng, counts, 2 * I, K, spare, aligned=aligned, lo=119, hi=121)
    h = torch.zeros(R, I, device="cuda")
    coli.mxfp4_swiglu(q, s, mats.table, I, mats.q_off, mats.s_off, offsets=off, out=h)
    hq = torch.full((R, I // 2), 0x5a, dtype=torch.uint8, device="cuda")
    hs = torch.full((R, I // 32), 0x5a, dtype=torch.uint8, device="cuda")
    got = coli.mxfp4_swiglu(q, s, mats.table, I, mats.q_off, mats.s_off, offsets=off, out=(hq, hs))
    assert got[0] is hq and got[1] is hs
    n = int(off_np[-1])
    qr, sr = coli.quantize_mxfp4(h[:n].contiguous())
    assert torch.equal(hs[:n], sr) and torch.equal(hq[:n], qr)
    assert bool((hq[n:] == 0x5a).all()) and bool((hs[n:] == 0x5a).all())
    q2, s2 = coli.mxfp4_swiglu(q, s, mats.table, I, mats.q_off, mats.s_off, offsets=off, dtype="mxfp4")
    assert torch.equal(q2[:n], hq[:n]) and torch.equal(s2[:n], hs[:n])


def test_swiglu_extreme_gates(coli):
    """Gates far on either side: silu goes to 0 and to the gate itself without NaN."""
    K, I = 32, 32
    gate = np.zeros((I, K))
    gate[:, 0] = np.where(np.arange(I) % 2, 6.0, -6.0)
    up = np.zeros((I, K))
    up[:, 0] = 1.0
    q, s = ref.quantize(ref.interleave(gate, up))
    blob = _dev(np.concatenate([q.ravel(), s.ravel()]))
    for mag in (1.0, 4.0, 2.0 ** 12, 2.0 ** 40):
        x = np.zeros((1, K))
        x[0, 0] = mag
        xq, xs = ref.quantize(x)
        h = _host(coli.mxfp4_swiglu(_dev(xq), _dev(xs), coli.blob_table([blob]), I, 0, I * K))
        g = gate[:, 0] * mag
        want = np.where(g > -700, g / (1 + np.exp(-np.maximum(g, -700))), 0.0) * mag
        assert (np.abs(h[0] - want) <= 16 * 2.0 ** -24 * np.abs(want) + 1e-30).all()


def test_quantize_expert_blob(coli):
    """An expert's blob holds the interleaved gate/up matrix and the down matrix as the products read them."""
    import torch
    rng = np.random.default_rng(11)
    shape = coli.MoEShape(160, 96, 2, top_k=1)
    H, I = shape.hidden, shape.inter
    off, nbytes = coli.mxfp4_blob_layout(shape)
    for dtype in DTYPES:
        g, u, d = (torch.from_numpy(rng.standard_normal(z) * 0.02).to(_t(dtype)) for z in ((I, H), (I, H), (H, I)))
        blob = coli.quantize_mxfp4_expert(shape, g.to("cuda"), u.to("cuda"), d.to("cuda")).cpu().numpy()
        assert blob.size == nbytes
        q, s = ref.quantize(ref.interleave(_host(g), _host(u)))
        assert np.array_equal(blob[off[0]:off[0] + I * H], q.ravel())
        assert np.array_equal(blob[off[2]:off[2] + 2 * I * H // 32], s.ravel())
        q, s = ref.quantize(_host(d))
        assert np.array_equal(blob[off[1]:off[1] + H * I // 2], q.ravel())
        assert np.array_equal(blob[off[3]:off[3] + H * I // 32], s.ravel())


def test_row_results_do_not_depend_on_other_rows(coli):
    """A row alone and among others (of the same count class or not) gives the same f32 sums where they are exact,
    and calls repeat bit for bit."""
    import torch
    rng = np.random.default_rng(2)
    mats, q, s, a, off, off_np, R = _case(coli, rng, [5, 0, 30, 1], 80, 1088, 0)
    args = (mats.table, 80, mats.q_off, mats.s_off)
    y = coli.mxfp4_matmul(q, s, *args, offsets=off)
    assert torch.equal(y, coli.mxfp4_matmul(q, s, *args, offsets=off))
    s2 = s.clone()
    s2[4] = 255                                                 # a neighbour of the same expert is NaN
    y2 = coli.mxfp4_matmul(q, s2, *args, offsets=off)
    assert torch.equal(y2[:4], y[:4]) and torch.equal(y2[5:], y[5:]) and bool(y2[4].isnan().all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_dequantize_every_scale(coli, dtype):
    """All 256 scale codes with all 16 element codes, the scales beyond the quantiser's (252) among them: 253 and 254
    pass f32 and bf16 from 2^128 on, to infinity."""
    import torch
    q = np.tile(np.arange(16, dtype=np.uint8) | np.arange(16, dtype=np.uint8) << 4, (256, 1))
    s = np.arange(256, dtype=np.uint8)[:, None]
    want = torch.from_numpy(ref.values(q, s)).to(_t(dtype))
    got = coli.dequantize_mxfp4(_dev(q), _dev(s), dtype=_t(dtype)).cpu()
    nan = want.isnan()
    assert bool(nan[255].all()) and not bool(nan[:255].any())
    assert torch.equal(got.isnan(), nan) and torch.equal(got[:255], want[:255])
    assert torch.equal(torch.signbit(got[:255]), torch.signbit(want[:255]))
    assert bool(got[254].isinf().any()) and bool(got[253].isinf().any())
