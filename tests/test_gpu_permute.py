"""Token permutation: the sort with its inverse, dispatch, combine and their
gradients against plain 64-bit forms; the whole MXFP4 expert layer built of
them; streams, graphs and refused tensors.

Tolerances: copies are exact. A sum of k f32 products is off by at most (k + 2)
half-steps (2^-24) of the sum of its terms' sizes, a dot product by (additions in a
row + 2) of them; each result then by half a step of its type."""
import numpy as np
import pytest

from tests import mxfp4_refs as ref

pytestmark = pytest.mark.gpu
DTYPES = ("float32", "bfloat16", "float16")
U = 2.0 ** -24


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


def _idx(rng, T, k, E, drop=0.0, repeat=False):
    if repeat:                                                  # the same expert twice in a token
        idx = rng.integers(0, E, (T, k))
    else:
        idx = np.argsort(rng.random((T, E)), 1)[:, :k]
    idx = np.where(rng.random((T, k)) < drop, rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], (T, k)), idx)
    return idx.astype(np.int32)


@pytest.mark.parametrize("T,k,E,drop", [(0, 2, 4, 0), (1, 1, 1, 0), (1, 8, 256, 0), (3, 4, 7, 0.5), (128, 8, 256, 0.1),
                                        (129, 8, 256, 0.1), (64, 16, 1024, 0.3), (1024, 1, 5, 0), (700, 3, 1024, 0.2),
                                        (5, 3, 9, 1.0), (2500, 8, 64, 0.05), (0, 2, 1020, 0), (9000, 8, 64, 0.05), (8192, 8, 1024, 0.01),
                                        (1023, 4, 256, 0.1), (512, 8, 470, 0.05), (512, 8, 480, 0.05), (4096, 1, 1, 0),
                                        (1025, 1, 1024, 0.1), (513, 8, 256, 0.1)])
def test_union_inverse(coli, T, k, E, drop):
    import torch
    rng = np.random.default_rng(T + k + E)
    idx = _idx(rng, T, k, E, drop, repeat=k > E or T % 2 == 1)
    counts, offsets, perm, unique, n_unique, inv = coli.union_inverse(_dev(idx), E)
    off_r, perm_r, inv_r = ref.sort(idx, E)
    n = int(off_r[-1])
    assert np.array_equal(offsets.cpu().numpy(), off_r)
    assert np.array_equal(counts.cpu().numpy(), np.diff(off_r))
    assert np.array_equal(perm.cpu().numpy()[:n], perm_r)
    assert np.array_equal(inv.cpu().numpy(), inv_r)
    used = np.nonzero(np.diff(off_r))[0]
    assert n_unique.item() == len(used) and np.array_equal(unique.cpu().numpy()[:len(used)], used)
    c2, o2, p2, u2, nu2 = coli.union(_dev(idx), E)              # the same answer as union
    assert torch.equal(c2, counts) and torch.equal(o2, offsets) and torch.equal(nu2, n_unique)
    assert torch.equal(p2[:n], perm[:n]) and torch.equal(u2[:len(used)], unique[:len(used)])


# T, k, E, H, share of slots without a row, row padding
CASES = [(1, 1, 1, 1, 0, 0), (1, 8, 16, 6144, 0, 0), (3, 2, 4, 7, 0.4, 0), (5, 3, 4, 33, 0.5, 3), (2, 4, 5, 64, 1.0, 0),
         (17, 5, 9, 2049, 0.2, 0), (40, 8, 32, 256, 0.1, 8), (9, 11, 16, 1000, 0.3, 1), (700, 4, 60, 96, 0.2, 0),
         (6, 32, 40, 4104, 0.2, 0), (11, 3, 6, 1002, 0.2, 0), (13, 6, 8, 514, 0.1, 2)]


def _setup(rng, T, k, E, H, drop, pad, dtype, n_mats):
    """inv, and n_mats (tensor with padded rows, 64-bit values) of T*k or T rows each."""
    import torch
    idx = _idx(rng, T, k, E, drop, repeat=T % 2 == 0)
    _, _, inv = ref.sort(idx, E)
    out = []
    for rows, kind in n_mats:
        x = torch.from_numpy(rng.standard_normal((rows, H))).to(_t(kind))
        buf = torch.full((rows, H + pad), float("nan"), dtype=_t(kind), device="cuda")
        buf[:, :H] = x.to("cuda")
        out.append((buf[:, :H], _host(x)))
    return inv, out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H,drop,pad", CASES)
def test_dispatch(coli, dtype, T, k, E, H, drop, pad):
    import torch
    rng = np.random.default_rng(T * 31 + H)
    inv, [(x, xr)] = _setup(rng, T, k, E, H, drop, pad, dtype, [(T, dtype)])
    buf = torch.full((T * k, H + pad), 7.0, dtype=_t(dtype), device="cuda")
    coli.dispatch(x, _dev(inv), out=buf[:, :H])
    want = np.full((T * k, H), 7.0)
    t, j = np.nonzero(inv >= 0)
    want[inv[t, j]] = xr[t]
    assert np.array_equal(_host(buf[:, :H]), want)
    assert bool((buf[:, H:] == 7.0).all())
    if H % 32 == 0:
        q = torch.full((T * k, H // 2), 0x5a, dtype=torch.uint8, device="cuda")
        s = torch.full((T * k, H // 32), 0x5a, dtype=torch.uint8, device="cuda")
        coli.dispatch_mxfp4(x, _dev(inv), q=q, s=s)
        qr, sr = ref.quantize(xr)
        wq, ws = np.full(q.shape, 0x5a, np.uint8), np.full(s.shape, 0x5a, np.uint8)
        wq[inv[t, j]], ws[inv[t, j]] = qr[t], sr[t]
        assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)


def test_dispatch_keeps_bits(coli):
    """NaN payloads and infinities are copied as they are."""
    import torch
    bits = torch.tensor([[0x7fc01234, 0x7f800000, -0x7fffff, 0x00000001, 0x7f812345]], dtype=torch.int32, device="cuda")
    inv = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    assert torch.equal(coli.dispatch(bits.view(torch.float32), inv).view(torch.int32), bits)
    half = bits.view(torch.int16)
    for kind in (torch.bfloat16, torch.float16):
        assert torch.equal(coli.dispatch(half.view(kind), inv).view(torch.int16), half)


@pytest.mark.parametrize("dtype,out", [("float32", "float32"), ("bfloat16", "bfloat16"), ("float16", "float16"),
                                       ("bfloat16", "float32"), ("float32", "float16"), ("float16", "bfloat16")])
@pytest.mark.parametrize("T,k,E,H,drop,pad", CASES)
def test_dispatch_bwd(coli, dtype, out, T, k, E, H, drop, pad):
    import torch
    rng = np.random.default_rng(T * 37 + H)
    inv, [(g, gr)] = _setup(rng, T, k, E, H, drop, pad, dtype, [(T * k, dtype)])
    gr = gr.copy()
    free = np.ones(T * k, bool)
    free[inv[inv >= 0]] = False
    g[torch.from_numpy(free).to("cuda")] = float("nan")         # rows of no slot: not read into any sum
    buf = torch.full((T, H + pad), 7.0, dtype=_t(out), device="cuda")
    coli.dispatch_bwd(g, _dev(inv), out=buf[:, :H])
    slots = ref.by_slot(gr, inv)
    want, size = slots.sum(1), np.abs(slots).sum(1)
    err = np.abs(_host(buf[:, :H]) - want)
    bound = (k + 2) * U * size
    assert (err <= bound + _half_step(out) * (np.abs(want) + bound)).all()
    assert bool((buf[:, H:] == 7.0).all())
    none = ~(inv >= 0).any(1)
    assert bool((buf[torch.from_numpy(none).to("cuda")][:, :H] == 0).all())


@pytest.mark.parametrize("rows_dtype,out", [("float32", "float32"), ("bfloat16", "bfloat16"), ("float16", "float16"),
                                            ("bfloat16", "float32"), ("float32", "bfloat16")])
@pytest.mark.parametrize("T,k,E,H,drop,pad", CASES)
@pytest.mark.parametrize("shared", [False, True])
def test_combine(coli, rows_dtype, out, T, k, E, H, drop, pad, shared):
    import torch
    rng = np.random.default_rng(T * 41 + H)
    inv, [(rows, rr), (sh, shr)] = _setup(rng, T, k, E, H, drop, pad, rows_dtype, [(T * k, rows_dtype), (T, out)])
    w = rng.standard_normal((T, k)).astype(np.float32)
    w[inv < 0] = np.nan                                          # the weight of a slot without a row is not used
    scale = 2.5
    buf = torch.full((T, H + pad), 7.0, dtype=_t(out), device="cuda")
    coli.combine(rows, _dev(inv), _dev(w), shared=sh if shared else None, scale=scale, out=buf[:, :H])
    wz = np.where(inv >= 0, w.astype(np.float64), 0.0)[..., None]
    terms = scale * wz * ref.by_slot(rr, inv)
    base = shr if shared else np.zeros((T, H))
    want, size = base + terms.sum(1), np.abs(base) + np.abs(terms).sum(1)
    bound = (k + 4) * U * size
    err = np.abs(_host(buf[:, :H]) - want)
    assert (err <= bound + _half_step(out) * (np.abs(want) + bound)).all()
    assert bool((buf[:, H:] == 7.0).all())
    if shared:                                                   # the output in the shared rows' place
        got = buf[:, :H].clone()
        coli.combine(rows, _dev(inv), _dev(w), shared=sh, scale=scale, out=sh)
        assert torch.equal(sh, got)


@pytest.mark.parametrize("dy_dtype,rows_dtype", [("float32", "float32"), ("bfloat16", "bfloat16"),
                                                 ("float16", "float16"), ("float32", "bfloat16"), ("bfloat16", "float32")])
@pytest.mark.parametrize("T,k,E,H,drop,pad", CASES)
def test_combine_bwd(coli, dy_dtype, rows_dtype, T, k, E, H, drop, pad):
    import torch
    rng = np.random.default_rng(T * 43 + H)
    inv, [(rows, rr), (dy, dyr)] = _setup(rng, T, k, E, H, drop, pad, rows_dtype, [(T * k, rows_dtype), (T, dy_dtype)])
    w = rng.standard_normal((T, k)).astype(np.float32)
    w[inv < 0] = np.nan
    scale = -1.75
    buf = torch.full((T * k, H + pad), 7.0, dtype=_t(rows_dtype), device="cuda")
    drows, dw = coli.combine_bwd(dy, rows, _dev(inv), _dev(w), scale=scale, rows_grad=buf[:, :H])
    want = np.full((T * k, H), 7.0)
    t, j = np.nonzero(inv >= 0)
    exact = scale * w[t, j].astype(np.float64)[:, None] * dyr[t]
    want[inv[t, j]] = exact
    err = np.abs(_host(buf[:, :H]) - want)
    bound = 2 * U * np.abs(want)
    assert (err <= bound + _half_step(rows_dtype) * (np.abs(want) + bound) + (2.0 ** -25 if rows_dtype == "float16" else 0)).all()
    assert bool((buf[:, H:] == 7.0).all())
    slots = scale * ref.by_slot(rr, inv) * dyr[:, None]
    adds = -(-H // 1024) * 8 + 12                                # in a lane's row, then over lanes and waves
    werr = np.abs(_host(dw) - slots.sum(2))
    assert (werr <= (adds + 2) * U * np.abs(slots).sum(2)).all()
    assert (_host(dw)[inv < 0] == 0).all()


def test_gradients_against_differences(coli):
    """combine is linear in the rows and in the weights, dispatch in x: differences of the forward calls, taken in
    64 bits over random directions, meet the gradients' inner products up to the f32 sums' rounding."""
    import torch
    rng = np.random.default_rng(9)
    T, k, E, H = 23, 4, 10, 515
    idx = _idx(rng, T, k, E, 0.2)
    inv = _dev(ref.sort(idx, E)[2])
    f = lambda *s: _dev(rng.standard_normal(s).astype(np.float32))
    rows, w, x, dy, g = f(T * k, H), f(T, k), f(T, H), f(T, H), f(T * k, H)
    used = torch.zeros(T * k, dtype=torch.bool, device="cuda")
    used[inv[inv >= 0].long()] = True
    rows[~used] = 0
    g[~used] = 0
    drows, dw = coli.combine_bwd(dy, rows, inv, w, scale=1.5, rows_grad=torch.zeros_like(rows))
    dx = coli.dispatch_bwd(g, inv)
    dot = lambda a, b: float((a.double() * b.double()).sum())
    size = lambda a, b: float((a.double() * b.double()).abs().sum())
    r_dir, w_dir, x_dir = f(T * k, H), f(T, k), f(T, H)
    r_dir[~used] = 0
    y = lambda r, v: coli.combine(r, inv, v, scale=1.5)
    # step 1: the call is linear along one input, so the difference has no remainder; the inputs' sums are rounded
    # to f32 first, and each call is off by at most (k + 4) U of its terms
    for up, down, want, terms in (
            (y(rows + r_dir, w), y(rows - r_dir, w), dot(drows, r_dir), 2 * size(y(rows.abs() + r_dir.abs(), w.abs()), dy)),
            (y(rows, w + w_dir), y(rows, w - w_dir), dot(dw, w_dir), 2 * size(y(rows.abs(), w.abs() + w_dir.abs()), dy))):
        got = (dot(up, dy) - dot(down, dy)) / 2
        assert abs(got - want) <= (H // 256 + 24 + k) * U * terms
    zero = torch.zeros(T * k, H, device="cuda")
    up, down = (coli.dispatch(x + s * x_dir, inv, out=zero.clone()) for s in (1, -1))
    assert abs((dot(up, g) - dot(down, g)) / 2 - dot(dx, x_dir)) <= (k + 8) * U * 2 * size(up.abs() + down.abs(), g)


def _expert_layer(coli, shape, x, idx, w, table, off, shared_table, rows_dtype):
    """One MXFP4 expert layer as a program runs it."""
    import torch
    H, I = shape.hidden, shape.inter
    _, offsets, _, _, _, inv = coli.union_inverse(idx, shape.n_routed)
    a = coli.dispatch_mxfp4(x, inv)
    h = coli.mxfp4_swiglu(*a, table, I, off[0], off[2], offsets=offsets, dtype="mxfp4")
    rows = coli.mxfp4_matmul(*h, table, H, off[1], off[3], offsets=offsets, dtype=rows_dtype)
    xq = coli.quantize_mxfp4(x)
    sh = coli.mxfp4_matmul(*coli.mxfp4_swiglu(*xq, shared_table, I, off[0], off[2], dtype="mxfp4"), shared_table, H,
                           off[1], off[3])
    return coli.combine(rows, inv, w, shared=sh, scale=shape.routed_scale, out=sh)


class Layer:
    def __init__(self, coli, seed, H, I, E, k):
        import torch
        rng = np.random.default_rng(seed)
        self.shape = coli.MoEShape(H, I, E, top_k=k, routed_scale=2.5)
        self.off = coli.mxfp4_blob_layout(self.shape)[0]
        self.mats, blobs = [], []
        for _ in range(E + 1):
            g, u, d = (rng.standard_normal(z).astype(np.float32) / 8 for z in ((I, H), (I, H), (H, I)))
            blobs.append(coli.quantize_mxfp4_expert(self.shape, _dev(g), _dev(u), _dev(d)))
            self.mats.append([ref.values(*ref.quantize(z)) for z in (g, u, d)])
        self.blobs = blobs
        self.table, self.shared = coli.blob_table(blobs[:E]), coli.blob_table(blobs[E:])

    def reference(self, x, idx, w):
        """The layer in 64 bits; h is quantised as the format defines."""
        xv = ref.values(*ref.quantize(x))

        def ffn(e, v):
            g, u, d = self.mats[e]
            a, b = v @ g.T, v @ u.T
            return ref.values(*ref.quantize(a / (1 + np.exp(-a)) * b)) @ d.T

        y = ffn(len(self.mats) - 1, xv)
        for e in range(self.shape.n_routed):
            t, j = np.nonzero(idx == e)
            if len(t):
                np.add.at(y, t, self.shape.routed_scale * w[t, j].astype(np.float64)[:, None] * ffn(e, xv[t]))
        return y

    def run(self, coli, x, idx, w, rows_dtype=None):
        return _expert_layer(coli, self.shape, x, idx, w, self.table, self.off, self.shared, rows_dtype)


@pytest.mark.parametrize("T,H,I,E,k,drop", [(1, 256, 128, 16, 4, 0), (7, 160, 96, 8, 2, 0.3), (70, 512, 256, 6, 3, 0.1),
                                            (400, 288, 160, 4, 2, 0)])
def test_expert_layer(coli, T, H, I, E, k, drop):
    """Router, sort, dispatch, both products and combine together. A 32-bit h next to a rounding border of the
    4-bit format may round the other way than the 64-bit h: at most a few of a layer's elements (an error of 1e-6
    of h against steps of at least a twelfth of it), each worth one step of one of `inter` terms."""
    import torch
    rng = np.random.default_rng(T)
    layer = Layer(coli, T, H, I, E, k)
    x = rng.standard_normal((T, H)).astype(np.float32)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    idx, w = coli.route(_dev(logits), None, k)
    if drop:
        gone = torch.from_numpy(rng.random((T, k)) < drop).to("cuda")
        idx, w = idx.masked_fill(gone, -1), w.masked_fill(gone, 0.0)
    y = layer.run(coli, _dev(x), idx, w)
    want = layer.reference(x, idx.cpu().numpy(), w.cpu().numpy())
    err = np.linalg.norm(_host(y) - want, axis=1) / np.linalg.norm(want, axis=1)
    # one flipped element of I moves a row by at most about 1 / (3 sqrt(I)) of its size; most rows have none
    assert np.median(err) <= 1e-5 and err.max() <= 1 / (3 * np.sqrt(I)), (float(np.median(err)), float(err.max()))


@pytest.mark.parametrize("T,H,I", [(40, 256, 128), (600, 1024, 1024), (90, 288, 544)])
def test_expert_layer_in_a_graph_and_on_streams(coli, T, H, I):
    """Captured calls replay to the eager result, with eager work between the replays; two graphs and a side stream
    run the same calls at once on outputs of their own. One case for each kernel of the products."""
    import torch
    rng = np.random.default_rng(3)
    layer = Layer(coli, 3, H, I, 8, 2)
    xs = [_dev(rng.standard_normal((T, H)).astype(np.float32)) for _ in range(3)]
    routes = [coli.route(_dev(rng.standard_normal((T, 8)).astype(np.float32)), None, 2) for _ in range(3)]
    want = [layer.run(coli, x, *r) for x, r in zip(xs, routes)]
    torch.cuda.synchronize()
    x, idx, w = xs[0].clone(), routes[0][0].clone(), routes[0][1].clone()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = layer.run(coli, x, idx, w)
        graphs.append(g)
        outs.append(out)
    side = torch.cuda.Stream()
    for rep in range(4):
        i = rep % 3
        x.copy_(xs[i]), idx.copy_(routes[i][0]), w.copy_(routes[i][1])
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            other = layer.run(coli, xs[(i + 1) % 3], *routes[(i + 1) % 3])
        for g in graphs:
            g.replay()
        eager = layer.run(coli, xs[i], *routes[i])
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[i]) for o in outs) and torch.equal(eager, want[i])
        assert torch.equal(other, want[(i + 1) % 3])


def test_gradients_in_a_graph(coli):
    """The backward calls captured and replayed while eager calls of the same tensors run between the replays."""
    import torch
    rng = np.random.default_rng(4)
    T, k, E, H = 33, 4, 12, 700
    idx = _dev(_idx(rng, T, k, E, 0.2))
    f = lambda *s: _dev(rng.standard_normal(s).astype(np.float32))
    rows, w, dy, g = f(T * k, H), f(T, k), f(T, H), f(T * k, H)
    drows = torch.zeros(T * k, H, device="cuda")

    def step():
        inv = coli.union_inverse(idx, E)[5]
        return coli.combine_bwd(dy, rows, inv, w, rows_grad=drows)[1], coli.dispatch_bwd(g, inv)

    want = [t.clone() for t in step()] + [drows.clone()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dw, dx = step()
    for _ in range(3):
        dw.zero_(), dx.zero_(), drows.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dw, want[0]) and torch.equal(dx, want[1]) and torch.equal(drows, want[2])
        got = step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_outputs_belong_to_the_given_stream(coli):
    """An output that a call allocates is the given stream's: when it is dropped, the current stream does not get its
    memory, where the call may still be writing. And the results are those of the current stream."""
    import torch
    rng = np.random.default_rng(6)
    T, k, H = 64, 4, 2048
    x, w = _dev(rng.standard_normal((T, H)).astype(np.float32)), _dev(rng.standard_normal((T, k)).astype(np.float32))
    rows = _dev(rng.standard_normal((T * k, H)).astype(np.float32))
    idx = _dev(np.stack([rng.permutation(16)[:k] for _ in range(T)]).astype(np.int32))   # every row is written
    inv = coli.union_inverse(idx, 16)[5]
    q, s = coli.quantize_mxfp4(rows)
    layer = Layer(coli, 1, H, 512, 1, 1)
    gu = layer.off[0], layer.off[2]
    shape = coli.MoEShape(128, 128, 1, top_k=1)                          # a blob without gaps
    gate = _dev(rng.standard_normal((128, 128)).astype(np.float32))
    calls = [
        lambda st: coli.quantize_mxfp4(x, stream=st), lambda st: coli.dequantize_mxfp4(q, s, stream=st),
        lambda st: coli.quantize_mxfp4_expert(shape, gate, gate, gate, stream=st),
        lambda st: coli.mxfp4_swiglu(q, s, layer.table, 512, *gu, stream=st),
        lambda st: coli.mxfp4_swiglu(q, s, layer.table, 512, *gu, dtype="mxfp4", stream=st),
        lambda st: coli.mxfp4_matmul(q, s, layer.table, 512, *gu, stream=st),
        lambda st: coli.union_inverse(idx, 16, stream=st), lambda st: coli.dispatch(x, inv, stream=st),
        lambda st: coli.dispatch_mxfp4(x, inv, stream=st), lambda st: coli.dispatch_bwd(rows, inv, stream=st),
        lambda st: coli.combine(rows, inv, w, stream=st), lambda st: coli.combine_bwd(x, rows, inv, w, stream=st)]
    side = torch.cuda.Stream()
    as_tuple = lambda o: o if isinstance(o, tuple) else (o,)
    for call in calls:
        want = [o.clone() for o in as_tuple(call(None))]
        torch.cuda.synchronize()
        got = as_tuple(call(side))
        torch.cuda.synchronize()
        meta = [(o.data_ptr(), o.numel() * o.element_size()) for o in got]
        for o, v in zip(got, want):
            assert torch.equal(o, v)
        del got, o
        for at, n in meta:
            held = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(8)]
            assert all(not at <= h.data_ptr() < at + n for h in held)


def test_stream_of_another_device_is_refused(coli):
    import torch

    class Other:
        device_index, cuda_stream = 1, 0

    x, out = torch.zeros(2, 64, device="cuda"), torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError, match="stream on device 1"):
        coli.dispatch(x, torch.zeros(2, 2, dtype=torch.int32, device="cuda"), out=out, stream=Other())


def test_places_outside_the_rows_are_skipped(coli):
    """Entries of inv below 0 or at least T*k mark slots without a row, whatever their value."""
    import torch
    inv = torch.tensor([[0, 4], [-7, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    x = torch.ones(2, 40, device="cuda")
    out = coli.dispatch(x, inv, out=torch.zeros(4, 40, device="cuda"))
    assert out.sum().item() == 40
    rows = torch.full((4, 40), 2.0, device="cuda")
    y = coli.combine(rows, inv, torch.ones(2, 2, device="cuda"))
    assert (y[0] == 2).all() and (y[1] == 0).all()


def test_binding_refuses_what_the_calls_cannot_take(coli):
    import torch
    x = torch.zeros(4, 64, device="cuda")
    inv = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    bad = [
        lambda: coli.quantize_mxfp4(x.t()),                              # columns not contiguous
        lambda: coli.quantize_mxfp4(x[:, :40]),                          # 40 columns
        lambda: coli.quantize_mxfp4(x[:1].expand(4, 64)),                # rows that overlap
        lambda: coli.quantize_mxfp4(x.double()),
        lambda: coli.quantize_mxfp4(x, q=torch.zeros(3, 32, dtype=torch.uint8, device="cuda")),
        lambda: coli.dequantize_mxfp4(torch.zeros(4, 32, dtype=torch.uint8, device="cuda"),
                                      torch.zeros(4, 3, dtype=torch.uint8, device="cuda")),
        lambda: coli.dispatch(x, inv.long()),
        lambda: coli.dispatch(x[:3], inv),                               # fewer tokens than inv
        lambda: coli.dispatch(x, inv, out=torch.zeros(7, 64, device="cuda")),
        lambda: coli.dispatch(x, inv, out=torch.zeros(8, 64, device="cuda", dtype=torch.float16)),
        lambda: coli.combine(torch.zeros(7, 64, device="cuda"), inv, w),
        lambda: coli.combine(torch.zeros(8, 64, device="cuda"), inv, w[:3]),
        lambda: coli.combine(torch.zeros(8, 64, device="cuda"), inv, w, shared=x[:, :32]),
        lambda: coli.combine_bwd(x[:, :32], torch.zeros(8, 64, device="cuda"), inv, w),
        lambda: coli.dispatch(x.cpu(), inv),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    q, s = coli.quantize_mxfp4(x)
    table = torch.zeros(2, dtype=torch.int64, device="cuda")
    for f in (lambda: coli.mxfp4_matmul(q, s, table, 8, offsets=torch.zeros(2, dtype=torch.int32, device="cuda")),
              lambda: coli.mxfp4_matmul(q, s, table.int(), 8),
              lambda: coli.mxfp4_swiglu(q, s, table, 48, dtype="mxfp4"),
              lambda: coli.mxfp4_swiglu(q, s, table[:1], 32, dtype=torch.float32,
                                        out=coli.quantize_mxfp4(x[:, :32])),
              lambda: coli.mxfp4_matmul(q, s, table[:1], 8, q_off=-16),
              lambda: coli.mxfp4_matmul(q, s, table[:1], 8, s_off=-16),
              lambda: coli.mxfp4_matmul(q, s, table[:1], 2 ** 32 + 8, out=torch.zeros(4, 8, device="cuda")),
              lambda: coli.mxfp4_matmul(q, s, table[:1], 8, out=torch.zeros(4, 9, device="cuda"))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(coli.ColiError):
        coli.mxfp4_matmul(q, s, table, 8)                                # two matrices need offsets


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("extra", [0, 3])
@pytest.mark.parametrize("side", [False, True])
def test_combine_bwd_own_rows_grad_is_zero_where_no_slot_is(coli, dtype, extra, side):
    """The rows' gradient that the call allocates itself: 0 in the rows that no slot has (whatever its memory held),
    and what a given buffer gets in the others."""
    import torch
    rng = np.random.default_rng(12)
    T, k, E, H = 19, 4, 9, 1026
    inv = _dev(ref.sort(_idx(rng, T, k, E, 0.4), E)[2])
    rows = _dev(rng.standard_normal((T * k + extra, H))).to(_t(dtype))
    dy, w = _dev(rng.standard_normal((T, H))).to(_t(dtype)), _dev(rng.standard_normal((T, k)).astype(np.float32))
    want, dw = coli.combine_bwd(dy, rows, inv, w, rows_grad=torch.zeros_like(rows))
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if side else None
    with torch.cuda.stream(stream):
        held = torch.full_like(rows, float("nan"))              # the memory that the next tensor of this size gets
        del held
    got, got_w = coli.combine_bwd(dy, rows, inv, w, stream=stream)
    torch.cuda.synchronize()
    used = torch.zeros(len(rows), dtype=torch.bool, device="cuda")
    used[inv[inv >= 0].long()] = True
    assert int((~used).sum()) > extra                            # some slots have no row
    assert bool((got[~used] == 0).all()) and torch.equal(got, want) and torch.equal(got_w, dw)


def test_inputs_of_a_given_stream_are_kept_until_it_is_done(coli):
    """A tensor that is dropped right after a call on another stream than its own: the current stream does not get its
    memory while the call has still to read (or write) it."""
    import torch
    rng = np.random.default_rng(8)
    T, k, H = 64, 4, 2048
    f = lambda *s: _dev(rng.standard_normal(s).astype(np.float32))
    x, rows, w, sh = f(T, H), f(T * k, H), f(T, k), f(T, H)
    idx = _dev(np.stack([rng.permutation(16)[:k] for _ in range(T)]).astype(np.int32))
    offsets, inv = coli.union_inverse(idx, 16)[1::4]
    q, s = coli.quantize_mxfp4(rows)
    layer = Layer(coli, 1, H, 128, 16, 1)
    gu = layer.off[0], layer.off[2]
    calls = [
        ([x], lambda a, st: coli.quantize_mxfp4(a, stream=st)), ([q, s], lambda a, b, st: coli.dequantize_mxfp4(a, b, stream=st)),
        ([q, s, layer.table, offsets], lambda a, b, c, d, st: coli.mxfp4_matmul(a, b, c, 128, *gu, offsets=d, stream=st)),
        ([q, s, layer.table, offsets], lambda a, b, c, d, st: coli.mxfp4_swiglu(a, b, c, 128, *gu, offsets=d, dtype="mxfp4", stream=st)),
        ([idx], lambda a, st: coli.union_inverse(a, 16, stream=st)), ([x, inv], lambda a, b, st: coli.dispatch(a, b, stream=st)),
        ([x, inv], lambda a, b, st: coli.dispatch_mxfp4(a, b, stream=st)),
        ([rows, inv], lambda a, b, st: coli.dispatch_bwd(a, b, stream=st)),
        ([rows, inv, w, sh], lambda a, b, c, d, st: coli.combine(a, b, c, shared=d, stream=st)),
        ([x, torch.zeros_like(x)], lambda a, o, st: (coli.dispatch(a, inv[:T // k], out=o, stream=st), ())[1]),   # a given output
        ([x, rows, inv, w], lambda a, b, c, d, st: coli.combine_bwd(a, b, c, d, stream=st))]
    side, square = torch.cuda.Stream(), torch.zeros(4096, 4096, device="cuda")
    as_tuple = lambda o: o if isinstance(o, tuple) else (o,)
    for tensors, call in calls:
        want = [o.clone() for o in as_tuple(call(*tensors, None))]
        own = [t.clone() for t in tensors]
        spans = [(t.data_ptr(), t.numel() * t.element_size()) for t in own]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):                                  # some 20 ms of work in front of the call
                square @ square
        got = as_tuple(call(*own, side))
        del own
        held = [[torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(4)] for _, n in spans]
        running = not side.query()
        for at, n in spans:
            for h in sum(held, []):
                assert at + n <= h.data_ptr() or h.data_ptr() + h.numel() <= at
        torch.cuda.synchronize()
        assert running
        for o, v in zip(got, want):
            assert torch.equal(o, v)


def test_given_stream_inside_a_capture(coli):
    """A captured program that forks into a stream of its own, drops the input and joins again."""
    import torch
    rng = np.random.default_rng(10)
    T, k, E, H = 50, 3, 8, 640
    x = _dev(rng.standard_normal((T, H)).astype(np.float32))
    inv = coli.union_inverse(_dev(_idx(rng, T, k, E, 0.0)), E)[5]
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        t = x * 2
        side.wait_stream(here)
        rows = coli.dispatch(t, inv, stream=side)
        del t
        other = x * 3                                            # would get t's memory
        here.wait_stream(side)
        return rows, other

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        eager = step()
        torch.cuda.synchronize()
        assert torch.equal(eager[0], want[0]) and torch.equal(eager[1], want[1])


def test_permutation_past_32_bits(coli):
    """Rows of more than 2^32 elements (9 GB): tokens at either end and in the middle meet the definition."""
    import torch
    T, k, H = 70_000, 8, 8192
    assert T * k * H > 2 ** 32 and T * k * H // 2 > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(5)
    inv = torch.randperm(T * k, device="cuda", generator=g).to(torch.int32).view(T, k)
    inv[T // 2, 3] = -1
    at = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    x = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    rows = coli.dispatch(x, inv)
    for t in at.tolist():
        for j in range(k):
            p = int(inv[t, j])
            assert p < 0 or torch.equal(rows[p], x[t])
    far = int(inv.argmax())                                      # the last row
    assert int(inv.view(-1)[far]) == T * k - 1 and torch.equal(rows[-1], x[far // k])
    q, s = coli.dispatch_mxfp4(x, inv)
    qt, st = coli.quantize_mxfp4(x[far // k][None])
    assert torch.equal(q[-1], qt[0]) and torch.equal(s[-1], st[0])
    del q, s
    kept = (inv[at] >= 0).unsqueeze(2)
    got = torch.where(kept, rows[inv[at].clamp_min(0).long()].double(), 0.0)             # [5][k][H]
    dx = coli.dispatch_bwd(rows, inv, dtype=torch.float32)
    assert ((dx[at].double() - got.sum(1)).abs() <= (k + 2) * U * got.abs().sum(1)).all()
    w = torch.rand(T, k, device="cuda", generator=g)
    y = coli.combine(rows, inv, w, dtype=torch.float32)
    terms = w[at].double().unsqueeze(2) * got
    assert ((y[at].double() - terms.sum(1)).abs() <= (k + 4) * U * terms.abs().sum(1)).all()
    drows, dw = coli.combine_bwd(x, rows, inv, w)
    for t in at.tolist():
        for j in range(k):
            p = int(inv[t, j])
            assert p < 0 or torch.equal(drows[p], (w[t, j] * x[t].float()).to(torch.bfloat16))
    slots = got * x[at].double().unsqueeze(1)
    adds = -(-H // 1024) * 8 + 12
    assert ((dw[at].double() - slots.sum(2)).abs() <= (adds + 2) * U * slots.abs().sum(2)).all()
    assert float(dw[T // 2, 3]) == 0
