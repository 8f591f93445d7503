"""Every kernel of the MXFP4 products, named before it runs, against plain 64-bit forms; and as a layer in graphs and
on two streams.

Scales lie within two binades on each side, so that every partial sum has at most 24 bits (test_gpu_mxfp4.py's
exactness test): products have one right answer in f32, whatever the order, and its rounding in the 16-bit types.
SwiGLU's gate and up sums are exact too; what follows is off by at most 16 half-steps of f32 (exp, add, divide,
two products), and 1e-37 below f32's range."""
import numpy as np
import pytest

from tests import mxfp4_cases as cases
from tests import mxfp4_refs as ref
from tests.test_gpu_mxfp4 import _case, _host, _t
from tests.test_gpu_permute import _expert_layer

pytestmark = pytest.mark.gpu
DTYPES = ("float32", "bfloat16", "float16")


@pytest.fixture(scope="module")
def coli():
    import int4_routed_expert_sigmoid_amd as c
    c.lib()
    return c


def _setup(coli, kernel, counts, K, aligned, spare, N):
    assert cases.chosen(coli, counts, spare, K, N, aligned) == kernel
    rng = np.random.default_rng(N * 31 + K)
    mats, q, s, a, off, off_np, R = _case(coli, rng, counts, N, K, spare, aligned=aligned, lo=119, hi=121)
    y = np.zeros((int(off_np[-1]), N))
    for e, m in enumerate(mats.values):
        y[off_np[e]:off_np[e + 1]] = a[off_np[e]:off_np[e + 1]] @ m.T
    return mats, q, s, off, R, y


@pytest.mark.parametrize("kernel,counts,K,aligned,spare", cases.CASES)
def test_matmul(coli, kernel, counts, K, aligned, spare):
    import torch
    N = cases.matrix_rows(kernel, counts, False)
    mats, q, s, off, R, want = _setup(coli, kernel, counts, K, aligned, spare, N)
    n = len(want)
    for dtype in DTYPES:
        for pad in (0, 5):                                      # rows of the output on any boundary
            buf = torch.full((R, N + pad), 7.0, dtype=_t(dtype), device="cuda")
            y = coli.mxfp4_matmul(q, s, mats.table, N, mats.q_off, mats.s_off, offsets=off, out=buf[:, :N])
            assert torch.equal(y[:n].cpu(), torch.from_numpy(want).to(_t(dtype))), (dtype, pad)
            assert bool((buf[:, N:] == 7.0).all()) and bool((buf[n:] == 7.0).all())


@pytest.mark.parametrize("kernel,counts,K,aligned,spare", cases.CASES)
def test_swiglu(coli, kernel, counts, K, aligned, spare):
    import torch
    I = cases.matrix_rows(kernel, counts, True)
    mats, q, s, off, R, gu = _setup(coli, kernel, counts, K, aligned, spare, 2 * I)
    n = len(gu)
    gu = gu.reshape(n, -1, 2, 16)
    g, u = gu[:, :, 0].reshape(n, I), gu[:, :, 1].reshape(n, I)
    want = g / (1 + np.exp(-g)) * u
    args = (q, s, mats.table, I, mats.q_off, mats.s_off)
    buf = torch.full((R, I + 3), 7.0, device="cuda")
    h = coli.mxfp4_swiglu(*args, offsets=off, out=buf[:, :I])
    err = np.abs(_host(h)[:n] - want)
    assert (err <= 16 * 2.0 ** -24 * np.abs(want) + 1e-37).all()
    assert bool((buf[:, I:] == 7.0).all()) and bool((buf[n:] == 7.0).all())
    for dtype in DTYPES[1:]:                                    # the f32 h, rounded once
        buf = torch.full((R, I + 3), 7.0, dtype=_t(dtype), device="cuda")
        got = coli.mxfp4_swiglu(*args, offsets=off, out=buf[:, :I])
        assert torch.equal(got[:n], h[:n].to(_t(dtype)))
        assert bool((buf[:, I:] == 7.0).all()) and bool((buf[n:] == 7.0).all())
    hq = torch.full((R, I // 2), 0x5a, dtype=torch.uint8, device="cuda")
    hs = torch.full((R, I // 32), 0x5a, dtype=torch.uint8, device="cuda")
    coli.mxfp4_swiglu(*args, offsets=off, out=(hq, hs))
    qr, sr = coli.quantize_mxfp4(h[:n])
    assert torch.equal(hs[:n], sr) and torch.equal(hq[:n], qr)
    assert bool((hq[n:] == 0x5a).all()) and bool((hs[n:] == 0x5a).all())


GROUPED = {c[0]: c for c in cases.CASES if not isinstance(c[1], int)}.values()   # the last one of each kernel


@pytest.mark.parametrize("kernel,counts,K,aligned,spare", GROUPED)
def test_a_share_of_the_experts(coli, kernel, counts, K, aligned, spare):
    """Offsets and table of some of the experts, as a rank that has them passes: the rows before the first offset and
    behind the last are neither read (they hold NaN) nor written."""
    import torch
    N, I = cases.matrix_rows(kernel, counts, False), cases.matrix_rows(kernel, counts, True)
    for n, swiglu in ((N, False), (2 * I, True)):
        rng = np.random.default_rng(K)
        mats, q, s, a, off, off_np, R = _case(coli, rng, [7] + counts + [11], n, K, 0, aligned=aligned, lo=119, hi=121)
        assert coli.debug_mxfp4_kernel(R, K, len(counts), n, True, aligned) == kernel
        lo, hi = int(off_np[1]), int(off_np[-2])
        args = (n if not swiglu else I, mats.q_off, mats.s_off)
        call = coli.mxfp4_swiglu if swiglu else coli.mxfp4_matmul
        want = call(q, s, mats.table, *args, offsets=off)
        s[:lo], s[hi:] = 255, 255
        out = torch.full((R, args[0]), 7.0, device="cuda")
        call(q, s, mats.table[1:-1], *args, offsets=off[1:-1], out=out)
        assert torch.equal(out[lo:hi], want[lo:hi]) and bool((out[:lo] == 7.0).all()) and bool((out[hi:] == 7.0).all())


@pytest.mark.parametrize("T,E,k,H,I,up,down", cases.LAYERS)
def test_layer_in_graphs_and_on_streams(coli, T, E, k, H, I, up, down):
    """A layer whose two products run the named kernels: captured calls replay to the eager result, with eager work
    between the replays, while a side stream runs the same calls on other inputs."""
    import torch
    assert coli.debug_mxfp4_kernel(T * k, H, E, 2 * I) == up and coli.debug_mxfp4_kernel(T * k, I, E, H) == down
    g = torch.Generator(device="cuda").manual_seed(T + H)
    shape = coli.MoEShape(H, I, E, top_k=k, routed_scale=2.5)
    off, size = coli.mxfp4_blob_layout(shape)
    blobs = torch.randint(0, 256, (E + 1, size), dtype=torch.uint8, device="cuda", generator=g)
    blobs[:, off[2]:] = blobs[:, off[2]:] % 3 + 118             # scales of weights near 0.02
    table = blobs.data_ptr() + size * torch.arange(E + 1, dtype=torch.int64)
    routed, shared = table[:E].cuda(), table[E:].cuda()
    xs = [torch.randn(T, H, device="cuda", generator=g) for _ in range(3)]
    routes = [coli.route(torch.randn(T, E, device="cuda", generator=g), None, k) for _ in range(3)]
    layer = lambda x, idx, w: _expert_layer(coli, shape, x, idx, w, routed, off, shared, None)
    want = [layer(x, *r) for x, r in zip(xs, routes)]
    torch.cuda.synchronize()
    assert all(bool(v.isfinite().all()) and float(v.abs().max()) > 0 for v in want)
    x, idx, w = xs[0].clone(), routes[0][0].clone(), routes[0][1].clone()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer(x, idx, w)
        graphs.append(graph)
        outs.append(out)
    side = torch.cuda.Stream()
    for rep in range(4):
        i = rep % 3
        x.copy_(xs[i]), idx.copy_(routes[i][0]), w.copy_(routes[i][1])
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            other = layer(xs[(i + 1) % 3], *routes[(i + 1) % 3])
        for graph in graphs:
            graph.replay()
        eager = layer(xs[i], *routes[i])
        torch.cuda.synchronize()
        assert all(torch.equal(o, want[i]) for o in outs) and torch.equal(eager, want[i])
        assert torch.equal(other, want[(i + 1) % 3])


def _random_rows(g, rows, K, lo):
    import torch
    q = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda").random_(0, 256, generator=g)
    return q, torch.randint(lo, lo + 2, (rows, K // 32), dtype=torch.uint8, device="cuda", generator=g)


@pytest.mark.parametrize("kernel,R,N,K", [("lines_256", 1_060_000, 40, 8192), ("lines_128", 33, 1_060_003, 8192),
                                          ("few_rows_4", 2, 1_060_003, 8192), ("tiles_128", 1_060_000, 40, 8160),
                                          ("tiles_128", 33, 1_060_003, 8160), ("tiles_short", 2_100, 1_060_003, 224),
                                          ("lines_256", 2_100, 1_060_003, 1024)])
def test_products_past_32_bits(coli, kernel, R, N, K):
    """Rows, matrices and outputs of more than 2^32 bytes: the last rows and columns are those of a call on them alone."""
    import torch
    assert coli.debug_mxfp4_kernel(R, K, 1, N, False) == kernel
    assert max(R * K // 2, N * K // 2, 2 * R * N) > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(N)
    a, a_s = _random_rows(g, R, K, 126)
    w, w_s = _random_rows(g, N, K, 119)
    r, n = min(R, 30), min(N, 35)
    blob = torch.cat([w.view(-1), w_s.view(-1)])
    del w, w_s
    table, s_off = coli.blob_table([blob]), N * K // 2
    y = coli.mxfp4_matmul(a, a_s, table, N, 0, s_off, dtype=torch.bfloat16)
    part = coli.mxfp4_matmul(a[-r:].clone(), a_s[-r:].clone(), table, n, (N - n) * (K // 2), s_off + (N - n) * (K // 32),
                             dtype=torch.bfloat16)               # sums are exact: any kernel gives the same
    assert torch.equal(y[-r:, -n:], part) and float(part.abs().max()) > 0
    first = coli.mxfp4_matmul(a[:r].clone(), a_s[:r].clone(), table, n, 0, s_off, dtype=torch.bfloat16)
    assert torch.equal(y[:r, :n], first) and not torch.equal(first, part)
