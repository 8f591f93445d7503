"""Routing with groups, and its gradient, against plain 64-bit forms.

Choices are equal to the reference's. Weights: the scores are within 2^-24 of the 64-bit ones (one rounding, and the
double exponential's), so are their double sums, and the weight is rounded once: 3 * 2^-24. Gradients are f32: exp, sums of
k or E terms, about 16 roundings of 2^-24 and one for every doubling of a wave's sum; bounded by 2^-18 of the largest
|term| of the row, plus the output type's half step."""
import numpy as np
import pytest

from tests import fp8_refs as ref

pytestmark = pytest.mark.gpu
DTYPES = ("float32", "bfloat16", "float16")


@pytest.fixture(scope="module")
def coli():
    import int4_routed_expert_sigmoid_amd as c
    c.lib()
    return c


def _t(name):
    import torch
    return getattr(torch, name)


def _inputs(T, E, dtype, seed, masked):
    import torch
    g = torch.Generator().manual_seed(seed)
    l = 1.5 * torch.randn(T, E, generator=g)
    if masked:
        l[torch.rand(T, generator=g) < 0.2] = -float("inf")
        l[torch.rand(T, E, generator=g) < 0.3] = -float("inf")
    l[torch.rand(T, E, generator=g) < 0.1] = 0.75                # equal keys where the bias is equal too
    b = 0.1 * torch.randn(E, generator=g)
    b[::3] = 0.0
    return l.to(_t(dtype)), b


CASES = [  # T, E, k, groups, kept, group_top
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (3, 2, 2, 2, 2, 2), (5, 2, 1, 2, 1, 2), (7, 60, 4, 4, 2, 2), (9, 63, 5, 7, 3, 1),
    (11, 64, 32, 64, 40, 2), (33, 72, 6, 8, 3, 2), (17, 129, 8, 3, 2, 2), (64, 160, 6, 8, 3, 1), (130, 256, 8, 8, 4, 2),
    (31, 320, 9, 5, 2, 2), (10, 512, 10, 16, 4, 2), (5, 513, 4, 27, 5, 1), (6, 1024, 32, 64, 8, 2), (4, 1000, 8, 1, 1, 1)]


@pytest.mark.parametrize("masked", (False, True))
@pytest.mark.parametrize("kind", ("sigmoid", "softmax"))
@pytest.mark.parametrize("T,E,k,groups,kept,top", CASES)
def test_route_matches_reference(coli, T, E, k, groups, kept, top, kind, masked):
    import torch
    for i, dtype in enumerate(DTYPES):
        l, b = _inputs(T, E, dtype, 100 * T + E + i, masked)
        norm = (T + i) % 2 == 0
        bias = None if (T + i) % 3 == 0 else b
        want_idx, want_w, s = ref.route(l.double().numpy(), None if bias is None else bias.numpy(), k, kind, groups, kept, top, norm, 2.5)
        idx, w, scores = coli.route_groups(l.cuda(), None if bias is None else bias.cuda(), k, score=kind, groups=groups,
                                           groups_kept=kept, group_top=top, norm=norm, scale=2.5, with_scores=True)
        assert np.array_equal(idx.cpu().numpy(), want_idx)
        assert np.abs(scores.cpu().numpy().astype(np.float64) - s).max() <= 2.0 ** -24
        assert (np.abs(w.cpu().numpy() - want_w) <= 3 * 2.0 ** -24 * np.abs(want_w)).all()
        i2, w2 = coli.route_groups(l.cuda(), None if bias is None else bias.cuda(), k, score=kind, groups=groups,
                                   groups_kept=kept, group_top=top, norm=norm, scale=2.5)
        assert torch.equal(i2, idx) and torch.equal(w2, w)


def test_one_group_is_the_plain_router(coli):
    """Sigmoid scores, one group: coli_moe_route's choice and weights, bit for bit."""
    import torch
    l, b = _inputs(77, 256, "float32", 3, False)
    idx, w = coli.route(l.cuda(), b.cuda(), 8)
    i2, w2 = coli.route_groups(l.cuda(), b.cuda(), 8)
    i3, w3 = coli.route_groups(l.cuda(), b.cuda(), 8, groups=8, groups_kept=8)
    assert torch.equal(idx, i2) and torch.equal(w, w2) and torch.equal(idx, i3) and torch.equal(w, w3)


def test_rows_that_masks_leave_empty(coli):
    """-infinity in every place, in all but one, in the bias; scores that are all 0; infinities and NaN."""
    import torch
    inf = float("inf")
    l = torch.zeros(7, 8)
    l[0] = -inf
    l[1] = -inf
    l[1, 5] = 1.0
    l[2] = -1e4                                                   # sigmoid scores of 0: equal shares
    l[3, 2] = float("nan")
    l[4, 6] = inf
    l[5, :4] = -inf
    b = torch.zeros(8)
    b[7] = -inf
    for kind in ("sigmoid", "softmax"):
        idx, w = coli.route_groups(l.cuda(), b.cuda(), 3, score=kind, groups=2, groups_kept=1)
        idx, w = idx.cpu(), w.cpu()
        assert idx[0].tolist() == [-1] * 3 and w[0].tolist() == [0.0] * 3
        assert idx[1].tolist() == [5, -1, -1] and w[1].tolist() == [1.0, 0.0, 0.0]
        assert idx[2].tolist() == [0, 1, 2] and torch.allclose(w[2], torch.full((3,), 1 / 3))
        for t in (3, 4):                                          # in range and distinct whatever the numbers are
            row = idx[t].tolist()
            assert len(set(row)) == 3 and all(0 <= e < 8 for e in row)
        assert idx[3, 0].item() in (2, 0) and bool(w[3].isnan().any())
        assert bool(w[4].isnan().any()) == (kind == "softmax")
        assert idx[5].tolist() == [4, 5, 6] and 7 not in idx.flatten().tolist()
        g = coli.route_groups_bwd(torch.ones(7, 3).cuda(), l.cuda(), idx.cuda(), score=kind, scores_grad=torch.ones(7, 8).cuda()).cpu()
        assert (g[0] == 0).all() and (g[1, [0, 1, 2, 3, 4, 6, 7]] == 0).all() and bool(torch.isfinite(g[[0, 1, 2, 5]]).all())
        c = coli.union(idx.cuda(), 8)[0].cpu()                    # the slots without expert reach no expert
        assert int(c.sum()) == int((idx >= 0).sum())


@pytest.mark.parametrize("kind", ("sigmoid", "softmax"))
@pytest.mark.parametrize("T,E,k,groups,kept,top", CASES)
def test_gradient_matches_formula(coli, T, E, k, groups, kept, top, kind):
    import torch
    for i, dtype in enumerate(DTYPES):
        l, b = _inputs(T, E, dtype, 7 * T + E + i, i == 1)
        norm = (T + i) % 2 == 0
        idx, _ = coli.route_groups(l.cuda(), b.cuda(), k, score=kind, groups=groups, groups_kept=kept, group_top=top)
        g = torch.Generator().manual_seed(T)
        gw, gs = torch.randn(T, k, generator=g), None if i == 2 else torch.randn(T, E, generator=g)
        want = ref.route_grad(gw.numpy(), l.double().numpy(), idx.cpu().numpy(), kind, norm, 2.5, None if gs is None else gs.numpy())
        for out in (dtype, "float32"):
            got = coli.route_groups_bwd(gw.cuda(), l.cuda(), idx, score=kind, norm=norm, scale=2.5,
                                        scores_grad=None if gs is None else gs.cuda(), dtype=_t(out))
            assert got.dtype == _t(out)
            got = got.double().cpu().numpy()
            most = 2.5 * np.abs(gw.numpy()).max(1, keepdims=True) + (0 if gs is None else np.abs(gs.numpy()).max(1, keepdims=True))
            bound = 2.0 ** -18 * most + torch.finfo(_t(out)).eps / 2 * np.abs(want) + torch.finfo(_t(out)).tiny
            assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("kind", ("sigmoid", "softmax"))
@pytest.mark.parametrize("E", (5, 96, 256, 320, 1024))
def test_masks_of_the_lowest_value(coli, E, kind):
    """Rows masked by their type's lowest finite value: all of them (softmax: equal scores), all but one place, together with
    -infinity, and values next to the lowest. Tolerances as for other rows."""
    import torch
    k = 4
    for dtype in DTYPES:
        low = torch.finfo(_t(dtype)).min
        l = _inputs(8, E, dtype, E, False)[0]
        l[0] = low
        l[1] = low
        l[1, E // 2] = 0.5
        l[2] = low
        l[2, ::2] = -float("inf")
        l[3] = low * 0.9995
        l[4, : E - 1] = low
        l[5, 1:] = low
        l[6] = -float("inf")
        gw, gs = torch.randn(8, k, generator=torch.Generator().manual_seed(E)), torch.randn(8, E, generator=torch.Generator().manual_seed(E + 1))
        for norm in (True, False):
            want_idx, want_w, s = ref.route(l.double().numpy(), None, k, kind, 1, 1, 1, norm, 2.5)
            idx, w, scores = coli.route_groups(l.cuda(), None, k, score=kind, norm=norm, scale=2.5, with_scores=True)
            assert np.array_equal(idx.cpu().numpy(), want_idx)
            assert np.abs(scores.cpu().numpy().astype(np.float64) - s).max() <= 2.0 ** -24
            assert (np.abs(w.cpu().numpy() - want_w) <= 3 * 2.0 ** -24 * np.abs(want_w)).all()
            if kind == "softmax":
                assert abs(scores[0, 0].item() * E - 1) < 1e-6
            want = ref.route_grad(gw.numpy(), l.double().numpy(), want_idx, kind, norm, 2.5, gs.numpy())
            got = coli.route_groups_bwd(gw.cuda(), l.cuda(), idx, score=kind, norm=norm, scale=2.5, scores_grad=gs.cuda(),
                                        dtype=torch.float32).double().cpu().numpy()
            most = 2.5 * np.abs(gw.numpy()).max(1, keepdims=True) + np.abs(gs.numpy()).max(1, keepdims=True)
            assert (np.abs(got - want) <= 2.0 ** -18 * most + 2.0 ** -24 * np.abs(want)).all()


# (64 of 8, 320 of 5, 512 of 16: a group is a power of two of whole lanes; the others': not)
@pytest.mark.parametrize("top", (1, 2))
@pytest.mark.parametrize("E,groups", ((64, 8), (320, 5), (512, 16), (60, 6), (72, 8), (336, 7)))
def test_groups_whose_keys_add_up_past_the_lowest(coli, E, groups, top):
    """A bias of f32's lowest value switches whole groups off, whose two keys together lie below it: they come after the
    others and before groups without any expert, and fill the slots that the others leave."""
    import torch
    size = E // groups
    k = min(32, size + 4)
    l = _inputs(9, E, "float32", E, False)[0]
    b = torch.full((E,), torch.finfo(torch.float32).min)
    b[:size] = -float("inf")                                      # no expert
    live = [size + 1, size + 3]
    b[size:2 * size] = -float("inf")
    b[live] = 0.0
    s = ref.scores(l.double().numpy(), "sigmoid").astype(np.float32)
    for norm in (True, False):
        idx, w = coli.route_groups(l.cuda(), b.cuda(), k, groups=groups, groups_kept=3, group_top=top, norm=norm)
        for t in range(9):
            first = sorted(live, key=lambda e: (-s[t, e], e))
            want = first + list(range(2 * size, 2 * size + k - 2))   # equal keys: the lower expert, and the lower group
            assert idx[t].tolist() == want
            got = s[t, want].astype(np.float64)
            got = got / got.sum() if norm else got
            assert (np.abs(w[t].cpu().numpy() - got) <= 3 * 2.0 ** -24 * got).all()


@pytest.mark.parametrize("kind", ("sigmoid", "softmax"))
@pytest.mark.parametrize("E,groups", ((8, 1), (64, 8), (72, 8), (320, 5)))
def test_a_bias_that_is_not_a_number(coli, E, groups, kind):
    """It comes first and shows in its slot's weight, with norm in all of the token's; a -infinity logit still takes its expert out."""
    import torch
    l = _inputs(6, E, "float32", E, False)[0]
    l[5, 3] = -float("inf")
    b = torch.zeros(E)
    b[3] = float("nan")
    plain = coli.route_groups(l.cuda(), None, 3, score=kind, with_scores=True)[2]
    for norm in (True, False):
        idx, w, scores = coli.route_groups(l.cuda(), b.cuda(), 3, score=kind, groups=groups, groups_kept=groups // 2 or 1, norm=norm,
                                           with_scores=True)
        assert idx[:5, 0].tolist() == [3] * 5 and bool(w[:5, 0].isnan().all())
        assert bool(w[:5, 1:].isnan().all()) if norm else bool(torch.isfinite(w[:5, 1:]).all())
        assert 3 not in idx[5].tolist() and bool(torch.isfinite(w[5]).all())
        assert torch.equal(scores, plain)


def test_gradient_of_small_scores_and_repeated_experts(coli):
    """Scores whose sum is near the smallest numbers keep the gradient of their shares; an expert named twice has both slots'."""
    import torch
    l = torch.full((2, 6), -90.0)
    l[1] = torch.tensor([0.5, -0.5, 1.0, 0.0, 2.0, -1.0])
    idx = torch.tensor([[0, 1], [2, 2]], dtype=torch.int32)
    gw = torch.tensor([[1.0, -1.0], [0.5, 1.5]])
    got = coli.route_groups_bwd(gw.cuda(), l.cuda(), idx.cuda()).double().cpu().numpy()
    want = ref.route_grad(gw.numpy(), l.double().numpy(), idx.numpy(), "sigmoid", True, 1.0)
    assert np.abs(got[0] - want[0]).max() <= 2.0 ** -8 and abs(got[0, 0] - 0.5) <= 2.0 ** -8     # subnormal scores: few bits
    got = coli.route_groups_bwd(gw.cuda(), l.cuda(), idx.cuda(), norm=False).double().cpu().numpy()
    want = ref.route_grad(gw.numpy(), l.double().numpy(), idx.numpy(), "sigmoid", False, 1.0)
    assert np.abs(got - want).max() <= 2.0 ** -20


def test_graph_stream_and_refusals(coli):
    import torch
    l, b = (x.cuda() for x in _inputs(50, 256, "bfloat16", 9, True))
    gw = torch.randn(50, 8, device="cuda")
    idx, w, s = coli.route_groups(l, b, 8, groups=8, groups_kept=4, with_scores=True)
    dl = coli.route_groups_bwd(gw, l, idx)
    outs = [torch.zeros_like(t) for t in (idx, w, s, dl)]

    def step(stream=None):
        coli.route_groups(l, b, 8, groups=8, groups_kept=4, idx=outs[0], w=outs[1], scores=outs[2], stream=stream)
        coli.route_groups_bwd(gw, l, outs[0], out=outs[3], stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(outs, (idx, w, s, dl)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        l.copy_(_inputs(50, 256, "bfloat16", 20 + seed, True)[0])
        graph.replay()
        torch.cuda.synchronize()
        idx, w, s = coli.route_groups(l, b, 8, groups=8, groups_kept=4, with_scores=True)
        assert all(torch.equal(a, c) for a, c in zip(outs, (idx, w, s, coli.route_groups_bwd(gw, l, idx))))
    for bad in (lambda: coli.route_groups(l.t(), b, 8), lambda: coli.route_groups(l, b[:5], 8), lambda: coli.route_groups(l, b.half(), 8),
                lambda: coli.route_groups(l, b, 8, score="tanh"), lambda: coli.route_groups(l.int(), b, 8),
                lambda: coli.route_groups(l, b, 8, idx=torch.empty(50, 7, dtype=torch.int32, device="cuda")),
                lambda: coli.route_groups_bwd(gw[:, :4], l, idx), lambda: coli.route_groups_bwd(gw, l, idx, out=dl[:5])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(coli.ColiError):
        coli.route_groups(l, b, 8, groups=8, groups_kept=0)
    i0, w0 = coli.route_groups(l[:0], b, 8)
    assert i0.shape == (0, 8) and coli.route_groups_bwd(w0, l[:0], i0).shape == (0, 256)


def test_many_tokens(coli):
    """More values than 2^31 bytes of scores: the last row lands where it belongs."""
    import torch
    T, E = 600_000, 1024
    l = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    l[-1, 7], l[T // 2, 9] = 3.0, 2.0
    idx, w, s = coli.route_groups(l, None, 2, with_scores=True)
    assert idx[-1].tolist() == [7, 0] and idx[T // 2].tolist() == [9, 0] and idx[0].tolist() == [0, 1]
    assert int((idx != torch.tensor([0, 1], device="cuda", dtype=torch.int32)).any(1).sum()) == 2
    assert abs(s[-1, 7].item() - 1 / (1 + np.exp(-3.0))) < 1e-6
    d = coli.route_groups_bwd(torch.ones(T, 2, device="cuda"), l, idx, norm=False, dtype=torch.bfloat16)
    assert int((d != 0).sum()) == 2 * T and d[-1, 7].item() > 0
