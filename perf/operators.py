"""The MXFP4 expert products and the token permutation around them, as cases that can be timed and compared.

Where `own` is false `run` computes the operators from elementary torch operations in 32 bits; where it is true it makes
the calls of the framework. Five operators and their chain:

  quantize   rows -> E2M1 codes with one E8M0 scale per 32 columns, and back to the values they stand for
  matmul     y[r] = W_e(r) a[r] for MXFP4 rows sorted by expert and MXFP4 matrices
  swiglu     h[r] = silu(G_e(r) a[r]) * (U_e(r) a[r]), gate and up rows interleaved in blocks of 16
  dispatch   the assignments sorted by expert, the tokens' rows copied into that order, and the gradient of the copy
  combine    y[t] = shared[t] + scale * sum_j w[t, j] rows[place of (t, j)], and its gradients
  chain      the five of them as an expert layer of MXFP4 weights runs them
"""
import math

import torch

own = False

BLOCK = 32                       # columns that share a scale
GATE_UP = 16                     # rows of gate, then as many of up, in an interleaved matrix
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token's activations on the way into an expert product: latency only
        {"name": "quantize-token", "op": "quantize", "rows": 1, "cols": 6144, "dtype": "bf16"},
        # the down matrices of 16 experts being converted at load time
        {"name": "quantize-weights", "op": "quantize", "rows": 98304, "cols": 2048, "dtype": "f32"},
        # the down product of one decoded token: 8 of 256 experts, one row each
        {"name": "matmul-decode", "op": "matmul", "rows": 8, "experts": 256, "n": 6144, "k": 2048, "dtype": "f32"},
        # one shared matrix over a long prompt, an odd number of rows: bound by the matrix cores
        {"name": "matmul-dense", "op": "matmul", "rows": 8191, "experts": 1, "n": 8192, "k": 8192, "dtype": "bf16"},
        # the gate and up product of one decoded token
        {"name": "swiglu-decode", "op": "swiglu", "rows": 8, "experts": 256, "n": 2048, "k": 6144, "dtype": "f32"},
        # the gate and up product of a 2048-token prompt over all 256 experts: bound by reading the weights
        {"name": "swiglu-prefill", "op": "swiglu", "rows": 16384, "experts": 256, "n": 2048, "k": 6144, "dtype": "bf16"},
        # a 2048-token prompt on its way to the experts
        {"name": "dispatch-prefill", "op": "dispatch", "tokens": 2048, "hidden": 6144, "experts": 256, "top": 8,
         "dropped": False, "train": False, "dtype": "bf16"},
        # a training step's sort, copy and gradient at odd sizes, with slots that an expert top-p dropped
        {"name": "dispatch-train", "op": "dispatch", "tokens": 1023, "hidden": 2049, "experts": 60, "top": 4,
         "dropped": True, "train": True, "dtype": "f32"},
        # the sum over the experts of a small batch of decoded tokens
        {"name": "combine-decode", "op": "combine", "tokens": 8, "hidden": 6144, "experts": 256, "top": 8,
         "dropped": True, "train": False, "dtype": "f32"},
        # a training step's weighted sum and its gradients to the rows and to the router's weights
        {"name": "combine-train", "op": "combine", "tokens": 4096, "hidden": 6144, "experts": 256, "top": 8,
         "dropped": False, "train": True, "dtype": "bf16"},
        # one decoded token through the whole layer
        {"name": "chain-decode", "op": "chain", "tokens": 1, "hidden": 6144, "inter": 2048, "experts": 256, "top": 8},
        # a 509-token chunk of a prompt through the whole layer: about 16 rows an expert
        {"name": "chain-chunk", "op": "chain", "tokens": 509, "hidden": 6144, "inter": 2048, "experts": 256, "top": 8},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("quantize", "matmul", "swiglu", "dispatch", "combine", "chain"))
    dtype = rng.choice(("f32", "bf16", "f16"))
    if op == "quantize":
        cols = BLOCK * _spread(rng, 1, 256)
        return {"op": op, "rows": _spread(rng, 1, min(131072, 200_000_000 // cols)), "cols": cols, "dtype": dtype}
    if op in ("matmul", "swiglu"):
        experts = rng.choice((1, _spread(rng, 2, 256)))
        k = BLOCK * _spread(rng, 1, 256)
        most = 3_200_000_000 // (experts * k)
        n = _spread(rng, 1, min(8192, most)) if op == "matmul" else BLOCK * _spread(rng, 1, max(1, min(128, most // 64)))
        rows = _spread(rng, 1, max(1, min(8192, 500_000_000_000 // (n * k))))
        return {"op": op, "rows": rows, "experts": experts, "n": n, "k": k, "dtype": dtype}
    top = rng.randint(1, 8)
    experts = _spread(rng, max(2, top), 256)
    if op == "chain":
        hidden, inter = BLOCK * _spread(rng, 1, 192), BLOCK * _spread(rng, 1, 64)
        return {"op": op, "tokens": _spread(rng, 1, 1024), "hidden": hidden, "inter": inter, "experts": experts, "top": top}
    hidden = _spread(rng, 1, 8192)
    tokens = _spread(rng, 1, max(1, min(16384, 100_000_000 // (top * hidden))))
    return {"op": op, "tokens": tokens, "hidden": hidden, "experts": experts, "top": top, "dropped": rng.random() < 0.5,
            "train": rng.random() < 0.5, "dtype": dtype}


# ---------------------------------------------------------------- inputs

def _matrices(g, experts, n, k):
    """[experts] blobs of an MXFP4 [n][k] matrix each (codes, then scales on a 256-byte boundary) with their device
    table. Uniform codes are what normal weights give: with a block's largest value between 4 and 8 scales, the eight
    magnitudes are about equally likely. Scales are those of weights of a standard deviation near 0.02."""
    s_off = -(-n * k // 2 // 256) * 256
    size = s_off + -(-n * k // BLOCK // 256) * 256
    blobs = torch.empty((experts, size), dtype=torch.uint8, device="cuda")
    q, s = blobs[:, :n * k // 2], blobs[:, s_off:s_off + n * k // BLOCK]
    q.random_(0, 256, generator=g)
    s.random_(119, 122, generator=g)
    table = blobs.data_ptr() + size * torch.arange(experts, dtype=torch.int64)
    return {"blobs": blobs, "table": table.cuda(), "s_off": s_off, "n": n,
            "q": q.unflatten(1, (n, k // 2)), "s": s.unflatten(1, (n, k // BLOCK))}


def _codes(g, rows, cols):
    """Quantised activations of a standard deviation near 1."""
    q = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, device="cuda", generator=g)
    return q, torch.randint(125, 128, (rows, cols // BLOCK), dtype=torch.uint8, device="cuda", generator=g)


def _routing(g, case):
    """Experts of unequal popularity, distinct within a token; weights that sum to 1; with `dropped` each token keeps a
    prefix of its slots, as an expert top-p leaves them."""
    T, E, k = case["tokens"], case["experts"], case["top"]
    scores = torch.randn(T, E, device="cuda", generator=g) + 0.5 * torch.randn(E, device="cuda", generator=g)
    top, idx = scores.topk(k, dim=1)
    idx, w = idx.to(torch.int32), torch.sigmoid(top)
    if case.get("dropped"):
        kept = torch.randint(1, k + 1, (T, 1), device="cuda", generator=g)
        out = torch.arange(k, device="cuda") >= kept
        idx, w = idx.masked_fill(out, -1), w.masked_fill(out, 0.0)
    return idx, w / w.sum(1, keepdim=True)


def _sorted_places(idx, E):
    """offsets [E + 1] of the assignments sorted by expert, and each assignment's place [T][k] (-1: none)."""
    e = idx.reshape(-1).to(torch.int64)
    e = torch.where(e < 0, E, e)
    order = torch.argsort(e, stable=True)
    place = torch.empty_like(order).scatter_(0, order, torch.arange(e.numel(), device=e.device))
    place = torch.where(e == E, -1, place)
    offsets = torch.searchsorted(e[order], torch.arange(E + 1, device=e.device))
    return offsets.to(torch.int32), place.to(torch.int32).view_as(idx)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    kind = TYPES[case.get("dtype", "bf16")]
    st = {"case": case}
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        st["x"] = torch.randn(rows, cols, device="cuda", generator=g).to(kind)
        st["x"][:, cols // 2:cols // 2 + 2] *= 30                  # outlying columns, as activations have
    elif op in ("matmul", "swiglu"):
        R, E, n, k = case["rows"], case["experts"], case["n"], case["k"]
        st["a"], st["a_s"] = _codes(g, R, k)
        st["w"] = _matrices(g, E, n * (2 if op == "swiglu" else 1), k)
        if R <= E:                                                 # a token's experts are distinct
            e = torch.randperm(E, device="cuda", generator=g)[:R]
        else:
            e = torch.multinomial(torch.rand(E, device="cuda", generator=g) + 0.5, R, replacement=True, generator=g)
        counts = torch.bincount(e, minlength=E)
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        st["most"] = int(counts.max())
        st["out"] = torch.zeros(R, n, dtype=kind, device="cuda")
    else:
        T, H, k = case["tokens"], case["hidden"], case["top"]
        st["idx"], st["weights"] = _routing(g, case)
        offsets, place = _sorted_places(st["idx"], case["experts"])
        n = T * k
        if op == "dispatch":
            st["x"] = torch.randn(T, H, device="cuda", generator=g).to(kind)
            st["rows"] = torch.zeros(n, H, dtype=kind, device="cuda")
            if case["train"]:
                st["grad"] = torch.randn(n, H, device="cuda", generator=g).to(kind)
        elif op == "combine":
            st["place"] = place
            st["rows"] = torch.randn(n, H, device="cuda", generator=g).to(kind)
            st["shared"] = torch.randn(T, H, device="cuda", generator=g).to(kind)
            if case["train"]:
                st["grad"] = torch.randn(T, H, device="cuda", generator=g).to(kind)
                st["rows_grad"] = torch.zeros(n, H, dtype=kind, device="cuda")
        else:
            I = case["inter"]
            st["x"] = torch.randn(T, H, device="cuda", generator=g).to(kind)
            st["gate_up"] = _matrices(g, case["experts"], 2 * I, H)
            st["down"] = _matrices(g, case["experts"], H, I)
            st["most"] = int((offsets[1:] - offsets[:-1]).max())
    return st


SCALE = 2.5                      # of the routed sum at the combine


def run(st):
    return _framework(st) if own else _plain(st)


# ---------------------------------------------------------------- the framework's calls

def _framework(st):
    import int4_routed_expert_sigmoid_amd as coli
    case, op = st["case"], st["case"]["op"]
    if op == "quantize":
        q, s = coli.quantize_mxfp4(st["x"])
        return coli.dequantize_mxfp4(q, s, dtype=torch.bfloat16)
    if op == "matmul":
        w = st["w"]
        return coli.mxfp4_matmul(st["a"], st["a_s"], w["table"], w["n"], s_off=w["s_off"], offsets=st["offsets"], out=st["out"])
    if op == "swiglu":
        w = st["w"]
        return coli.mxfp4_swiglu(st["a"], st["a_s"], w["table"], case["n"], s_off=w["s_off"], offsets=st["offsets"], out=st["out"])
    if op == "dispatch":
        got = coli.union_inverse(st["idx"], case["experts"])
        offsets, inv = got[1], got[5]
        out = {"offsets": offsets, "place": inv, "rows": coli.dispatch(st["x"], inv, out=st["rows"])}
        if case["train"]:
            out["x_grad"] = coli.dispatch_bwd(st["grad"], inv)
        return out
    if op == "combine":
        out = {"y": coli.combine(st["rows"], st["place"], st["weights"], shared=st["shared"], scale=SCALE)}
        if case["train"]:
            out["rows_grad"], out["w_grad"] = coli.combine_bwd(st["grad"], st["rows"], st["place"], st["weights"], scale=SCALE,
                                                               rows_grad=st["rows_grad"])
        return out
    got = coli.union_inverse(st["idx"], case["experts"])
    offsets, inv = got[1], got[5]
    up, down = st["gate_up"], st["down"]
    a, a_s = coli.dispatch_mxfp4(st["x"], inv)
    h, h_s = coli.mxfp4_swiglu(a, a_s, up["table"], case["inter"], s_off=up["s_off"], offsets=offsets, dtype="mxfp4")
    rows = coli.mxfp4_matmul(h, h_s, down["table"], down["n"], s_off=down["s_off"], offsets=offsets, dtype=torch.bfloat16)
    return coli.combine(rows, inv, st["weights"], scale=SCALE)


# ---------------------------------------------------------------- the plain forms, in 32 bits

def _scale_values(s):
    """2^(s - 127); 255 stands for NaN."""
    s = s.to(torch.int32)
    bits = torch.where(s == 0, 1 << 22, s << 23)
    return torch.where(s == 255, 0x7fc00000, bits).view(torch.float32)


def _values(q, s):
    """The values of codes [..., K / 2] with scales [..., K / 32]."""
    one = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=q.device)
    pairs = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)              # by byte: low nibble, high nibble
    v = pairs[q.to(torch.int32)].view(*s.shape, BLOCK)
    return v.mul_(_scale_values(s).unsqueeze(-1)).view(*s.shape[:-1], -1)


def _quantized(x):
    """x [..., K] -> the values that its MXFP4 form stands for."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1)
    s = ((top.view(torch.int32) >> 23) - 2).clamp_min(0)
    a = b.abs() * ((254 - s) << 23).view(torch.float32).unsqueeze(-1)
    level = ((a > 0.25).to(torch.int32) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    v = torch.tensor(MAGNITUDES, device=x.device)[level] * _scale_values(s).unsqueeze(-1)
    return torch.copysign(v, b).flatten(-2)


def _product(a, w, offsets, most):
    """a [R][K] with the matrices' values, rows by expert; rows past the last offset are 0."""
    R, E = a.shape[0], offsets.numel() - 1
    offsets = offsets.to(torch.int64)
    row = torch.arange(R, device=a.device)
    e = torch.searchsorted(offsets[1:], row, right=True)
    used = (e < E).unsqueeze(1)
    e = e.clamp(max=E - 1)
    if R < E:                                                      # few rows: their experts' matrices alone
        y = torch.bmm(_values(w["q"][e], w["s"][e]), a.unsqueeze(2)).squeeze(2)
    else:
        place = (offsets[:-1, None] + torch.arange(most, device=a.device)).clamp(max=R - 1)
        y = torch.bmm(_values(w["q"], w["s"]), a[place].transpose(1, 2).contiguous())
        y = y[e, :, (row - offsets[e]).clamp(max=most - 1)]
    return y.where(used, 0.0)


def _swiglu(gu):
    gu = gu.unflatten(1, (-1, 2, GATE_UP))
    g, u = gu[:, :, 0].flatten(1), gu[:, :, 1].flatten(1)
    return g * torch.sigmoid(g) * u


def _rows_of(x, place):
    """x's rows at their tokens' places; rows of no place are 0."""
    n, k = place.numel(), place.shape[1]
    at = torch.where(place < 0, n, place).reshape(-1).to(torch.int64)
    return x.new_zeros(n + 1, x.shape[1]).index_copy_(0, at, x.repeat_interleave(k, 0))[:n]


def _by_slot(rows, place):
    """The rows [T][k][H] of every slot in 32 bits, 0 where it has none."""
    got = rows[place.clamp_min(0).to(torch.int64)].float()
    return got.masked_fill((place < 0).unsqueeze(2), 0.0)


def _plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "quantize":
        return _quantized(st["x"]).to(torch.bfloat16)
    if op in ("matmul", "swiglu"):
        y = _product(_values(st["a"], st["a_s"]), st["w"], st["offsets"], st["most"])
        return (_swiglu(y) if op == "swiglu" else y).to(st["out"].dtype)
    if op == "dispatch":
        offsets, place = _sorted_places(st["idx"], case["experts"])
        out = {"offsets": offsets, "place": place, "rows": _rows_of(st["x"], place)}
        if case["train"]:
            out["x_grad"] = _by_slot(st["grad"], place).sum(1).to(st["x"].dtype)
        return out
    if op == "combine":
        rows, w, kind = _by_slot(st["rows"], st["place"]), st["weights"], st["rows"].dtype
        y = st["shared"].float() + SCALE * (w.unsqueeze(2) * rows).sum(1)
        out = {"y": y.to(kind)}
        if case["train"]:
            g = st["grad"].float()
            slots = (SCALE * w.unsqueeze(2) * g.unsqueeze(1)).to(kind).flatten(0, 1)
            n = st["place"].numel()
            at = torch.where(st["place"] < 0, n, st["place"]).reshape(-1).to(torch.int64)
            out["rows_grad"] = slots.new_zeros(n + 1, slots.shape[1]).index_copy_(0, at, slots)[:n]
            out["w_grad"] = SCALE * (rows * g.unsqueeze(1)).sum(2)
        return out
    offsets, place = _sorted_places(st["idx"], case["experts"])
    a = _rows_of(_quantized(st["x"]), place)
    h = _swiglu(_product(a, st["gate_up"], offsets, st["most"]))
    rows = _product(_quantized(h), st["down"], offsets, st["most"]).to(torch.bfloat16)
    return (SCALE * (st["weights"].unsqueeze(2) * _by_slot(rows, place)).sum(1)).to(torch.bfloat16)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    held = 0.5 + 1 / BLOCK                                         # bytes of a value in MXFP4
    size = 4 if case.get("dtype") == "f32" else 2
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size + 2 * held + 2), "flops": 4 * n}
    if op in ("matmul", "swiglu"):
        R, E, n, k = case["rows"], case["experts"], case["n"], case["k"]
        rows = n * (2 if op == "swiglu" else 1)
        return {"bytes": R * k * held + min(E, R) * rows * k * held + R * n * size, "flops": 2 * R * rows * k}
    T, H, k = case["tokens"], case["hidden"], case["top"]
    n = T * k * (0.5 * (k + 1) / k if case.get("dropped") else 1)  # rows that have a place
    if op == "dispatch":
        once = T * H * size + n * H * size
        return {"bytes": 3 * T * k * 4 + once * (2 if case["train"] else 1), "flops": n * H}
    if op == "combine":
        bytes_ = T * k * 8 + (2 * T + n) * H * size
        if case["train"]:
            bytes_ += T * k * 8 + (T + 2 * n) * H * size
        return {"bytes": bytes_, "flops": n * H * (6 if case["train"] else 2)}
    I, E = case["inter"], case["experts"]
    hit = min(E, T * k)
    return {"bytes": 2 * T * H * 2 + hit * 3 * H * I * held + T * k * (H * held + 2 * I * held + 2 * H * 2),
            "flops": 2 * T * k * 3 * H * I}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _exact_values(q, s):
    codes = torch.stack([q & 15, q >> 4], -1).flatten(-2).to(torch.int32)
    e, m = (codes >> 1) & 3, (codes & 1).double()
    v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2((e - 1).double()).round())
    v = torch.where(codes >= 8, -v, v).unflatten(-1, (-1, BLOCK))
    return (v * torch.ldexp(torch.ones_like(s, dtype=torch.float64), s.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def _exact_quantized(x):
    b = x.double().unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    step = torch.ldexp(torch.ones_like(top), (torch.frexp(top).exponent - 3).clamp(-127, 127))
    a = (b / step).abs()
    a = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2))).clamp(max=6)
    return (torch.sign(b) * a * step).flatten(-2)


def _exact_product(a, w, offsets):
    y = a.new_zeros(a.shape[0], w["n"])
    ends = offsets.tolist()
    for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if hi > lo:
            y[lo:hi] = a[lo:hi] @ _exact_values(w["q"][e], w["s"][e]).t().contiguous()
    return y


def _exact_swiglu(gu):
    at = torch.arange(gu.shape[1] // 2, device=gu.device)
    at = at // GATE_UP * 2 * GATE_UP + at % GATE_UP
    g, u = gu[:, at], gu[:, at + GATE_UP]
    return g / (1 + torch.exp(-g)) * u


def _exact_slots(rows, place):
    return rows.double()[place.clamp_min(0).to(torch.int64)] * (place >= 0).unsqueeze(2)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantized(st["x"])
    if op in ("matmul", "swiglu"):
        y = _exact_product(_exact_values(st["a"], st["a_s"]), st["w"], st["offsets"])
        return _exact_swiglu(y) if op == "swiglu" else y
    idx = st["idx"]
    flat = idx.reshape(-1).tolist()
    order = sorted((e, a) for a, e in enumerate(flat) if e >= 0)
    place = torch.full((idx.numel(),), -1, dtype=torch.int32)
    place[torch.tensor([a for _, a in order], dtype=torch.int64)] = torch.arange(len(order), dtype=torch.int32)
    place = place.view(idx.shape).to(idx.device)
    counts = [0] * (case["experts"] + 1)
    for e, _ in order:
        counts[e + 1] += 1
    offsets = torch.tensor(counts, dtype=torch.int64).cumsum(0).to(torch.int32).to(idx.device)
    if op == "dispatch":
        rows = torch.zeros(idx.numel(), case["hidden"], dtype=torch.float64, device=idx.device)
        t, j = torch.nonzero(place >= 0, as_tuple=True)
        rows[place[t, j].to(torch.int64)] = st["x"].double()[t]
        out = {"offsets": offsets, "place": place, "rows": rows}
        if case["train"]:
            out["x_grad"] = _exact_slots(st["grad"], place).sum(1)
        return out
    w = st["weights"].double()
    if op == "combine":
        slots = _exact_slots(st["rows"], place)
        out = {"y": st["shared"].double() + SCALE * (w.unsqueeze(2) * slots).sum(1)}
        if case["train"]:
            g = st["grad"].double()
            t, j = torch.nonzero(place >= 0, as_tuple=True)
            out["rows_grad"] = torch.zeros(idx.numel(), case["hidden"], dtype=torch.float64, device=idx.device)
            out["rows_grad"][place[t, j].to(torch.int64)] = SCALE * w[t, j].unsqueeze(1) * g[t]
            out["w_grad"] = SCALE * (slots * g.unsqueeze(1)).sum(2)
        return out
    x = _exact_quantized(st["x"])
    a = x.new_zeros(idx.numel(), case["hidden"])
    t, j = torch.nonzero(place >= 0, as_tuple=True)
    a[place[t, j].to(torch.int64)] = x[t]
    h = _exact_swiglu(_exact_product(a, st["gate_up"], offsets))
    rows = _exact_product(_exact_quantized(h), st["down"], offsets)
    return SCALE * (w.unsqueeze(2) * _exact_slots(rows, place)).sum(1)
