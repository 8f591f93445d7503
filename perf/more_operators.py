"""Routing with groups, and expert products in 8-bit floating point with a scale for each block of 128, as cases that can
be timed and compared.

Where `own` is false `run` computes the operators from elementary torch operations in 32 bits (64 where a choice or a
rounding hangs on the last bit); where it is true it makes the calls of the framework. Five operators and their chain:

  route      softmax or sigmoid scores, a bias and groups for the selection, top-k, weights; and the logits' gradient
  quantize   rows (1 x 128 blocks) or matrices (128 x 128 blocks, both ways round) -> e4m3 codes and scales, and back
  matmul     y[r] = W_e(r) a[r], rows sorted by expert
  swiglu     h[r] = silu(G_e(r) a[r]) * (U_e(r) a[r])
  backward   of the product: the rows' gradient through the transposed matrices, and every matrix' gradient from rows and
             output gradients quantised over 128 rows of an expert
  chain      the expert layer of one batch: route, sort, dispatch, both products, combine
"""
import math

import torch

own = False

BLOCK = 128                      # columns (or rows and columns) that share a scale
LARGEST = 448.0                  # of e4m3
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SCALE = 2.5                      # of the router's weights


def listed():
    return [
        # one decoded token through the router: latency only
        {"name": "route-token", "op": "route", "tokens": 1, "experts": 256, "top": 8, "score": "sigmoid", "groups": 8,
         "kept": 4, "norm": True, "masked": False, "train": False, "dtype": "f32"},
        # a training batch with padded tokens, with the gradients of the weights and of a balance loss on the scores
        {"name": "route-train", "op": "route", "tokens": 16384, "experts": 256, "top": 8, "score": "softmax", "groups": 8,
         "kept": 4, "norm": True, "masked": True, "train": True, "dtype": "bf16"},
        # a prompt's rows on their way into the down product
        {"name": "quantize-rows", "op": "quantize", "kind": "rows", "count": 1, "rows": 16383, "cols": 2048, "dtype": "bf16"},
        # the down matrices of 16 experts after an optimiser step: for the product and for its gradient
        {"name": "quantize-matrices", "op": "quantize", "kind": "matrix", "count": 16, "rows": 6144, "cols": 2048, "dtype": "f32"},
        # the down product of one decoded token: 8 of 256 experts, one row each
        {"name": "matmul-decode", "op": "matmul", "rows": 8, "experts": 256, "n": 6144, "k": 2048, "dtype": "f32"},
        # one shared matrix over a long prompt, an odd number of rows: bound by the matrix cores
        {"name": "matmul-dense", "op": "matmul", "rows": 8191, "experts": 1, "n": 8192, "k": 8192, "dtype": "bf16"},
        # the gate and up product of one decoded token
        {"name": "swiglu-decode", "op": "swiglu", "rows": 8, "experts": 256, "n": 2048, "k": 6144, "dtype": "bf16"},
        # the gate and up product of a 2048-token prompt over all 256 experts
        {"name": "swiglu-prefill", "op": "swiglu", "rows": 16384, "experts": 256, "n": 2048, "k": 6144, "dtype": "f16"},
        # a training step's gradients of one matrix that every token goes through
        {"name": "backward-dense", "op": "backward", "rows": 4095, "experts": 1, "n": 6144, "k": 8192, "dtype": "bf16"},
        # a training step's gradients of 64 experts
        {"name": "backward-experts", "op": "backward", "rows": 16384, "experts": 64, "n": 2048, "k": 6144, "dtype": "bf16"},
        # one decoded token through the whole layer
        {"name": "chain-decode", "op": "chain", "tokens": 1, "hidden": 6144, "inter": 2048, "experts": 256, "top": 8,
         "groups": 8, "kept": 4},
        # a 509-token chunk of a prompt through the whole layer: about 16 rows an expert
        {"name": "chain-chunk", "op": "chain", "tokens": 509, "hidden": 6144, "inter": 2048, "experts": 256, "top": 8,
         "groups": 8, "kept": 4},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _groups(rng, experts, top):
    """(groups, kept) that leave at least `top` experts."""
    groups = rng.choice([g for g in (1, 2, 4, 8, 16) if experts % g == 0])
    least = -(-top // (experts // groups))
    return groups, rng.randint(least, groups)


def draw(rng):
    op = rng.choice(("route", "quantize", "matmul", "swiglu", "backward", "chain"))
    dtype = rng.choice(("f32", "bf16", "f16"))
    if op == "route":
        top = rng.randint(1, 8)
        experts = _spread(rng, max(2, top), 512)
        groups, kept = _groups(rng, experts, top)
        return {"op": op, "tokens": _spread(rng, 1, 4_000_000 // experts), "experts": experts, "top": top,
                "score": rng.choice(("sigmoid", "softmax")), "groups": groups, "kept": kept, "norm": rng.random() < 0.7,
                "masked": rng.random() < 0.5, "train": rng.random() < 0.5, "dtype": dtype}
    if op == "quantize":
        kind = rng.choice(("rows", "matrix"))
        cols = 16 * _spread(rng, 1, 512)
        if kind == "rows":
            return {"op": op, "kind": kind, "count": 1, "rows": _spread(rng, 1, min(131072, 100_000_000 // cols)),
                    "cols": cols, "dtype": dtype}
        rows = 16 * _spread(rng, 1, 512)
        return {"op": op, "kind": kind, "count": _spread(rng, 1, max(1, min(64, 100_000_000 // (rows * cols)))),
                "rows": rows, "cols": cols, "dtype": dtype}
    if op in ("matmul", "swiglu", "backward"):
        experts = rng.choice((1, _spread(rng, 2, 256)))
        k = 16 * _spread(rng, 1, 512)
        most = (800_000_000 if op == "backward" else 3_200_000_000) // (experts * k)
        if op == "matmul":
            n = _spread(rng, 1, min(8192, most))
        else:
            n = 16 * _spread(rng, 1, max(1, min(256, most // 32)))
        rows = _spread(rng, 1, max(1, min(8192, 200_000_000_000 // (n * k))))
        return {"op": op, "rows": rows, "experts": experts, "n": n, "k": k, "dtype": dtype}
    top = rng.randint(1, 8)
    experts = _spread(rng, max(2, top), 256)
    groups, kept = _groups(rng, experts, top)
    return {"op": op, "tokens": _spread(rng, 1, 500), "hidden": 16 * _spread(rng, 1, 384),
            "inter": 16 * _spread(rng, 1, 128), "experts": experts, "top": top, "groups": groups, "kept": kept}


# ---------------------------------------------------------------- inputs

def _ceil(n):
    return -(-n // BLOCK)


def _codes(g, *shape):
    """e4m3 codes of normal values, as a block's quantised ones are: the largest of 128 near the end of the range."""
    x = torch.randn(*shape, device="cuda", generator=g).mul_(110).clamp_(-LARGEST, LARGEST)
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _matrices(g, experts, n, k, two=False):
    """[experts] buffers of an FP8 [n][k] matrix each (codes, then the blocks' scales on a 256-byte boundary) with their
    device table; `two`: a gate and an up matrix of n rows each, codes and scales of one behind those of the other.
    Scales are those of weights of a standard deviation near 0.02, any 32-bit numbers as checkpoints have them."""
    parts = 2 if two else 1
    s_off = -(-parts * n * k // 256) * 256
    sn, sk = _ceil(n), _ceil(k)
    size = s_off + -(-4 * parts * sn * sk // 256) * 256
    blobs = torch.zeros((experts, size), dtype=torch.uint8, device="cuda")
    for e in range(experts):
        blobs[e, :parts * n * k] = _codes(g, parts * n * k)
        s = 2e-4 * (0.5 + torch.rand(parts * sn * sk, device="cuda", generator=g))
        blobs[e, s_off:s_off + 4 * parts * sn * sk] = s.view(torch.uint8)
    table = blobs.data_ptr() + size * torch.arange(experts, dtype=torch.int64)
    return {"blobs": blobs, "table": table.cuda(), "s_off": s_off, "n": n, "k": k, "parts": parts}


def _part(w, p, chosen=None):
    """(codes [experts][n][k], scales [experts][n / 128][k / 128]) of part p of the (chosen) matrices."""
    n, k, sn, sk = w["n"], w["k"], _ceil(w["n"]), _ceil(w["k"])
    blobs = w["blobs"] if chosen is None else w["blobs"][chosen]
    at = w["s_off"] + 4 * p * sn * sk
    return (blobs[:, p * n * k:(p + 1) * n * k].unflatten(1, (n, k)),
            blobs[:, at:at + 4 * sn * sk].contiguous().view(torch.float32).unflatten(1, (sn, sk)))


def _offsets(g, rows, experts):
    """offsets [experts + 1] of rows over experts of unequal popularity; few rows are a token's, of distinct experts."""
    if rows <= experts:
        e = torch.randperm(experts, device="cuda", generator=g)[:rows]
    else:
        e = torch.multinomial(torch.rand(experts, device="cuda", generator=g) + 0.5, rows, replacement=True, generator=g)
    counts = torch.bincount(e, minlength=experts)
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32), int(counts.max())


def _logits(g, case, kind):
    T, E = case["tokens"], case["experts"]
    x = 1.5 * torch.randn(T, E, device="cuda", generator=g) + 0.5 * torch.randn(E, device="cuda", generator=g)
    if case.get("masked"):                                         # padded tokens, and an expert that is switched off
        x[torch.rand(T, device="cuda", generator=g) < 0.1] = -math.inf
        x[:, E // 2] = -math.inf
    return x.to(kind)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    kind = TYPES[case.get("dtype", "bf16")]
    st = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top"]
        st["logits"], st["bias"] = _logits(g, case, kind), 0.1 * normal(E)
        if case["train"]:
            st["w_grad"], st["scores_grad"] = normal(T, k), 0.01 * normal(T, E)
    elif op == "quantize":
        shape = (case["rows"], case["cols"]) if case["kind"] == "rows" else (case["count"], case["rows"], case["cols"])
        st["x"] = normal(*shape).to(kind)
        st["x"][..., case["cols"] // 2:case["cols"] // 2 + 2] *= 30   # outlying columns, as activations have
    elif op in ("matmul", "swiglu", "backward"):
        R, E, n, k = case["rows"], case["experts"], case["n"], case["k"]
        st["offsets"], st["most"] = _offsets(g, R, E)
        if op == "backward":
            st["wt"] = _matrices(g, E, k, n)                       # the matrices the other way round
            st["x"], st["grad"] = normal(R, k).to(kind), (0.01 * normal(R, n)).to(kind)
        else:
            st["w"] = _matrices(g, E, n, k, two=op == "swiglu")
            st["a"] = _codes(g, R, k)
            st["a_s"] = torch.exp2(torch.randint(-8, -5, (R, _ceil(k)), device="cuda", generator=g).float())
            st["out"] = torch.zeros(R, n, dtype=kind, device="cuda")
    else:
        st["x"] = normal(case["tokens"], case["hidden"]).to(kind)
        st["logits"], st["bias"] = _logits(g, case, torch.float32), 0.1 * normal(case["experts"])
        st["gate_up"] = _matrices(g, case["experts"], case["inter"], case["hidden"], two=True)
        st["down"] = _matrices(g, case["experts"], case["hidden"], case["inter"])
    return st


def run(st):
    return _framework(st) if own else _plain(st)


# ---------------------------------------------------------------- the framework's calls

def _framework(st):
    import int4_routed_expert_sigmoid_amd as coli
    case, op = st["case"], st["case"]["op"]
    if op == "route":
        how = dict(score=case["score"], groups=case["groups"], groups_kept=case["kept"], norm=case["norm"], scale=SCALE)
        if not case["train"]:
            idx, w = coli.route_groups(st["logits"], st["bias"], case["top"], **how)
            return {"idx": idx, "w": w}
        idx, w, scores = coli.route_groups(st["logits"], st["bias"], case["top"], with_scores=True, **how)
        grad = coli.route_groups_bwd(st["w_grad"], st["logits"], idx, score=case["score"], norm=case["norm"], scale=SCALE,
                                     scores_grad=st["scores_grad"], dtype=torch.float32)
        return {"idx": idx, "w": w, "scores": scores, "logits_grad": grad}
    if op == "quantize":
        if case["kind"] == "rows":
            q, s = coli.quantize_fp8(st["x"])
            return coli.dequantize_fp8(q, s, dtype=torch.bfloat16)
        q, s, qt, s_t = coli.quantize_fp8_matrix(st["x"], transposed=True)
        return {"values": coli.dequantize_fp8(q, s, dtype=torch.bfloat16),
                "transposed": coli.dequantize_fp8(qt, s_t, dtype=torch.bfloat16)}
    if op == "matmul":
        w = st["w"]
        return coli.fp8_matmul(st["a"], st["a_s"], w["table"], w["n"], s_off=w["s_off"], offsets=st["offsets"], out=st["out"])
    if op == "swiglu":
        w = st["w"]
        return coli.fp8_swiglu(st["a"], st["a_s"], w["table"], w["n"], s_off=w["s_off"], offsets=st["offsets"], out=st["out"])
    if op == "backward":
        w, offsets = st["wt"], st["offsets"]
        gt, gt_s, g, g_s = coli.quantize_fp8_columns(st["grad"], offsets, rows=True)
        xt, xt_s = coli.quantize_fp8_columns(st["x"], offsets)
        return {"x_grad": coli.fp8_matmul(g, g_s, w["table"], w["n"], s_off=w["s_off"], offsets=offsets, dtype=st["x"].dtype),
                "w_grad": coli.fp8_wgrad(gt, gt_s, xt, xt_s, offsets, dtype=torch.float32)}
    idx, w = coli.route_groups(st["logits"], st["bias"], case["top"], groups=case["groups"], groups_kept=case["kept"],
                               scale=SCALE)
    got = coli.union_inverse(idx, case["experts"])
    offsets, inv = got[1], got[5]
    up, down = st["gate_up"], st["down"]
    a, a_s = coli.dispatch_fp8(st["x"], inv)
    h, h_s = coli.fp8_swiglu(a, a_s, up["table"], up["n"], s_off=up["s_off"], offsets=offsets, dtype="fp8")
    rows = coli.fp8_matmul(h, h_s, down["table"], down["n"], s_off=down["s_off"], offsets=offsets, dtype=torch.bfloat16)
    return {"idx": idx, "y": coli.combine(rows, inv, w)}


# ---------------------------------------------------------------- the plain forms, in 32 bits

def _route(logits, bias, k, score, groups, kept, norm):
    """(idx, w, scores): the scores in 64 bits rounded once, the selection's keys and sums of keys in 32."""
    T, E = logits.shape
    l = logits.double()
    if score == "sigmoid":
        s = (1 / (1 + torch.exp(-l))).float()
    else:
        top = l.amax(1, keepdim=True).clamp_min(-1e300)
        e = torch.exp(l - top)
        s = (e / e.sum(1, keepdim=True).clamp_min(1e-300)).float()
    there = (l > -math.inf) & (bias > -math.inf)
    key = torch.where(there, s + bias, -math.inf)
    if groups > 1:
        two = key.unflatten(1, (groups, -1)).sort(dim=2, descending=True)[0][:, :, :2]
        value = two[..., 0]
        if two.shape[2] > 1:
            value = torch.where(two[..., 1] > -math.inf, two[..., 0] + two[..., 1], value)
        order = value.sort(dim=1, descending=True, stable=True)[1][:, :kept]
        open_ = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order, True)
        key = torch.where(open_.repeat_interleave(E // groups, 1), key, -math.inf)
    best, idx = key.sort(dim=1, descending=True, stable=True)
    best, idx = best[:, :k], idx[:, :k]
    used = best > -math.inf
    w = s.gather(1, idx).double().masked_fill(~used, 0.0)
    if norm:
        total, n = w.sum(1, keepdim=True), used.sum(1, keepdim=True).clamp_min(1)
        w = torch.where(total > 0, w / total.clamp_min(1e-300), used / n.double())
    return idx.masked_fill(~used, -1).to(torch.int32), (SCALE * w).float(), s


def _route_grad(st, idx, norm, score):
    l, g = st["logits"].float(), st["w_grad"]
    used = idx >= 0
    at = idx.clamp_min(0).to(torch.int64)
    if score == "sigmoid":
        s = torch.sigmoid(l)
    else:
        e = torch.exp(l - l.amax(1, keepdim=True).clamp_min(-1e30))
        s = e / e.sum(1, keepdim=True).clamp_min(1e-30)
    sel = s.gather(1, at).masked_fill(~used, 0.0)
    g = SCALE * g.masked_fill(~used, 0.0)
    if norm:
        total = sel.sum(1, keepdim=True)
        share = sel / total.clamp_min(1e-30)
        g = torch.where(total > 0, (g - (g * share).sum(1, keepdim=True)) / total.clamp_min(1e-30), 0.0)
        g = g.masked_fill(~used, 0.0)
    ds = st["scores_grad"].scatter_add(1, at, g)
    if score == "sigmoid":
        return ds * s * torch.sigmoid(-l)
    return s * (ds - (ds * s).sum(1, keepdim=True))


def _power(top):
    """The smallest power of two, at least 2^-126, that brings `top` (32 bits) to 448 or less."""
    bits = top.view(torch.int32)
    e = (bits >> 23) - 8 + ((bits & 0x7fffff) > 0x600000).to(torch.int32)
    return (e.clamp_min(1) << 23).view(torch.float32)


def _e4m3(x):
    """x (at most 448 in size) rounded to e4m3, a tie to the even code."""
    return x.to(torch.float8_e4m3fn).float()


def _quantized(x):
    """x [..., K] -> the values that its FP8 form with a scale for 128 columns stands for."""
    k = x.shape[-1]
    b = torch.nn.functional.pad(x.float(), (0, -k % BLOCK)).unflatten(-1, (-1, BLOCK))
    s = _power(b.abs().amax(-1, keepdim=True))
    return (_e4m3(b * (1 / s)) * s).flatten(-2)[..., :k]


def _quantized_matrix(x):
    n, k = x.shape[-2:]
    b = torch.nn.functional.pad(x.float(), (0, -k % BLOCK, 0, -n % BLOCK)).unflatten(-2, (-1, BLOCK)).unflatten(-1, (-1, BLOCK))
    s = _power(b.abs().amax((-3, -1), keepdim=True))
    return (_e4m3(b * (1 / s)) * s).flatten(-2).flatten(-3, -2)[..., :n, :k]


def _values(q, s, rows=True):
    """The values of codes [..., N][K] with scales for 128 columns of a row, or of 128 rows."""
    n, k = q.shape[-2:]
    v = q.view(torch.float8_e4m3fn).float()
    s = s.repeat_interleave(BLOCK, -1)[..., :k]
    return v * (s if rows else s.repeat_interleave(BLOCK, -2)[..., :n, :])


def _by_expert(offsets, most, R):
    """Every expert's rows in a matrix of its own [E][most], rows past its last one as R."""
    lo, hi = offsets[:-1, None].to(torch.int64), offsets[1:, None].to(torch.int64)
    at = lo + torch.arange(most, device=offsets.device)
    return torch.where(at < hi, at, R)


def _product(a, w, offsets, most, p=0):
    """a [R][K] with the matrices' values, rows by expert; rows past the last offset are 0."""
    R, E = a.shape[0], offsets.numel() - 1
    row = torch.arange(R, device=a.device)
    e = torch.searchsorted(offsets[1:].to(torch.int64), row, right=True)
    used = (e < E).unsqueeze(1)
    e = e.clamp(max=E - 1)
    if R < E:                                                      # few rows: their experts' matrices alone
        y = torch.bmm(_values(*_part(w, p, e), rows=False), a.unsqueeze(2)).squeeze(2)
    else:
        place = _by_expert(offsets, most, R).clamp(max=R - 1)
        y = torch.bmm(_values(*_part(w, p), rows=False), a[place].transpose(1, 2).contiguous())
        y = y[e, :, (row - offsets[e]).clamp(max=most - 1)]
    return y.where(used, 0.0)


def _swiglu(a, w, offsets, most):
    gate = _product(a, w, offsets, most, 0)
    return gate * torch.sigmoid(gate) * _product(a, w, offsets, most, 1)


def _plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "route":
        idx, w, scores = _route(st["logits"], st["bias"], case["top"], case["score"], case["groups"], case["kept"], case["norm"])
        if not case["train"]:
            return {"idx": idx, "w": w}
        return {"idx": idx, "w": w, "scores": scores, "logits_grad": _route_grad(st, idx, case["norm"], case["score"])}
    if op == "quantize":
        if case["kind"] == "rows":
            return _quantized(st["x"]).to(torch.bfloat16)
        v = _quantized_matrix(st["x"]).to(torch.bfloat16)
        return {"values": v, "transposed": v.transpose(1, 2).contiguous()}
    if op == "matmul":
        return _product(_values(st["a"], st["a_s"]), st["w"], st["offsets"], st["most"]).to(st["out"].dtype)
    if op == "swiglu":
        return _swiglu(_values(st["a"], st["a_s"]), st["w"], st["offsets"], st["most"]).to(st["out"].dtype)
    if op == "backward":
        offsets, most, grad, x = st["offsets"], st["most"], st["grad"].float(), st["x"].float()
        place = _by_expert(offsets, _ceil(most) * BLOCK, grad.shape[0])
        by_expert = []
        for rows in (grad, x):                                     # [E][n][rows], a scale for 128 of an expert's rows
            cols = torch.cat([rows, rows.new_zeros(1, rows.shape[1])])[place].transpose(1, 2).contiguous()
            by_expert.append(_quantized(cols))
        return {"x_grad": _product(_quantized(grad), st["wt"], offsets, most).to(st["x"].dtype),
                "w_grad": torch.bmm(by_expert[0], by_expert[1].transpose(1, 2).contiguous())}
    idx, w, _ = _route(st["logits"], st["bias"], case["top"], "sigmoid", case["groups"], case["kept"], True)
    T, k, E = case["tokens"], case["top"], case["experts"]
    flat = idx.reshape(-1).to(torch.int64)
    order = torch.argsort(flat, stable=True)
    offsets = torch.searchsorted(flat[order], torch.arange(E + 1, device=flat.device)).to(torch.int32)
    most = int(torch.bincount(flat, minlength=E).max())
    a = _quantized(st["x"])[order // k]
    h = _quantized(_swiglu(a, st["gate_up"], offsets, most))
    rows = _product(h, st["down"], offsets, most).to(torch.bfloat16).float()
    back = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device=order.device))
    return {"idx": idx, "y": (w.unsqueeze(2) * rows[back].unflatten(0, (T, k))).sum(1).to(torch.bfloat16)}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    size = 4 if case.get("dtype") == "f32" else 2
    held = 1 + 4 / BLOCK                                           # bytes of a value with a scale for 128
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top"]
        bytes_, flops = T * E * size + 4 * E + T * k * 8, 30 * T * E
        if case["train"]:
            bytes_ += T * E * (4 + 4 + 4) + T * k * 4              # the scores, their gradient, the logits' gradient
            flops += 15 * T * E
        return {"bytes": bytes_, "flops": flops}
    if op == "quantize":
        n = case["count"] * case["rows"] * case["cols"]
        if case["kind"] == "rows":
            return {"bytes": n * (size + 2 * held + 2), "flops": 4 * n}
        return {"bytes": n * (size + 2 * (2 + 2)), "flops": 4 * n}
    if op in ("matmul", "swiglu"):
        R, E, n, k = case["rows"], case["experts"], case["n"], case["k"]
        wide = n * (2 if op == "swiglu" else 1)
        return {"bytes": R * k * held + min(E, R) * wide * k + R * n * size, "flops": 2 * R * wide * k}
    if op == "backward":
        R, E, n, k = case["rows"], case["experts"], case["n"], case["k"]
        return {"bytes": R * (n + k) * size + min(E, R) * n * k + R * k * size + E * n * k * 4, "flops": 4 * R * n * k}
    T, H, I, k, E = case["tokens"], case["hidden"], case["inter"], case["top"], case["experts"]
    return {"bytes": 2 * T * H * 2 + T * E * 4 + min(E, T * k) * 3 * H * I + T * k * (H * held + 2 * I * held + 2 * H * 2),
            "flops": 2 * T * k * 3 * H * I}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _exact_power(e):
    """2^e, by its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_decode(q):
    q = q.to(torch.int32)
    e, m = (q >> 3) & 15, (q & 7).double()
    v = torch.where(e == 0, m / 512, (1 + m / 8) * _exact_power(e - 7))
    return torch.where(q >= 128, -v, v)


def _exact_round(x):
    """x to e4m3: 4 significant bits, steps of 2^-9 at least, half to even."""
    step = _exact_power((torch.frexp(x).exponent - 4).clamp_min(-9))
    return torch.round(x / step) * step


def _exact_rows(x):
    """Quantised along the last dimension, block by block."""
    x = x.double().clone()
    for at in range(0, x.shape[-1], BLOCK):
        b = x[..., at:at + BLOCK]
        top = b.abs().amax(-1, keepdim=True)
        m, e = torch.frexp(top / LARGEST)                          # top / 448 = m 2^e, m in [0.5, 1)
        s = _exact_power(torch.where(m == 0.5, e - 1, e).clamp_min(-126))
        x[..., at:at + BLOCK] = _exact_round(b / s) * s
    return x


def _exact_matrix(x):
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for i in range(0, x.shape[-2], BLOCK):
        for j in range(0, x.shape[-1], BLOCK):
            b = x[..., i:i + BLOCK, j:j + BLOCK].double()
            out[..., i:i + BLOCK, j:j + BLOCK] = _exact_tile(b)
    return out


def _exact_tile(b):
    top = b.abs().amax((-2, -1), keepdim=True)
    m, e = torch.frexp(top / LARGEST)
    s = _exact_power(torch.where(m == 0.5, e - 1, e).clamp_min(-126))
    return _exact_round(b / s) * s


def _exact_weight(w, p, e):
    n, k = w["n"], w["k"]
    q, s = _part(w, p, slice(e, e + 1))
    at_n = torch.arange(n, device=q.device) // BLOCK
    at_k = torch.arange(k, device=q.device) // BLOCK
    return _exact_decode(q[0]) * s[0].double()[at_n][:, at_k]


def _exact_product(a, w, offsets, p=0):
    y = a.new_zeros(a.shape[0], w["n"])
    ends = offsets.tolist()
    for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
        if hi > lo:
            y[lo:hi] = a[lo:hi] @ _exact_weight(w, p, e).t().contiguous()
    return y


def _exact_swiglu(a, w, offsets):
    g = _exact_product(a, w, offsets, 0)
    return g / (1 + torch.exp(-g)) * _exact_product(a, w, offsets, 1)


def _exact_scores(logits, score):
    l = logits.double()
    if score == "sigmoid":
        return torch.sigmoid(l)
    s = torch.softmax(l, 1)
    return torch.where(torch.isneginf(l).all(1, keepdim=True), 0.0, s)


def _exact_route(logits, bias, k, score, groups, kept, norm):
    """Expert by expert: the rank of a key is how many keys come before it."""
    s = _exact_scores(logits, score)
    s32 = s.float()
    T, E = s.shape
    there = ~torch.isneginf(logits) & ~torch.isneginf(bias)
    key = torch.where(there, s32 + bias, float("-inf"))

    def ranks(v):
        n = v.shape[1]
        rank = torch.zeros(v.shape, dtype=torch.int32, device=v.device)
        for j in range(n):
            other = v[:, j:j + 1]
            rank += (other > v) | ((other == v) & (torch.arange(n, device=v.device) > j))
        return rank

    if groups > 1:
        of = key.view(T, groups, E // groups)
        first = of.amax(2)
        rest = of.scatter(2, of.argmax(2, keepdim=True), float("-inf")).amax(2)
        value = torch.where(torch.isneginf(rest), first, first + rest)
        closed = ranks(value) >= kept
        key = key.masked_fill(closed.repeat_interleave(E // groups, 1), float("-inf"))
    rank = ranks(key)
    taken = (rank < k) & ~torch.isneginf(key)
    idx = torch.full((T, k), -1, dtype=torch.int32, device=s.device)
    w = torch.zeros(T, k, dtype=torch.float64, device=s.device)
    t, e = torch.nonzero(taken, as_tuple=True)
    slot = rank[t, e].to(torch.int64)
    idx[t, slot] = e.to(torch.int32)
    w[t, slot] = s[t, e]
    if norm:
        total, n = w.sum(1, keepdim=True), (idx >= 0).sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, (idx >= 0) / n.clamp_min(1).double())
    return idx, SCALE * w, s


def _exact_route_grad(st, idx, s, norm, score):
    t, j = torch.nonzero(idx >= 0, as_tuple=True)
    e = idx[t, j].to(torch.int64)
    g = torch.zeros(idx.shape, dtype=torch.float64, device=s.device)
    g[t, j] = SCALE * st["w_grad"].double()[t, j]
    if norm:
        sel = torch.zeros_like(g)
        sel[t, j] = s[t, e]
        total = sel.sum(1, keepdim=True)
        g = torch.where(total > 0, (g - (g * sel).sum(1, keepdim=True) / total) / total, 0.0)
    ds = st["scores_grad"].double().clone()
    ds[t, e] += g[t, j]
    if score == "sigmoid":
        return ds * s * torch.sigmoid(-st["logits"].double())
    return s * (ds - (s * ds).sum(1, keepdim=True))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        idx, w, s = _exact_route(st["logits"], st["bias"], case["top"], case["score"], case["groups"], case["kept"], case["norm"])
        if not case["train"]:
            return {"idx": idx, "w": w}
        return {"idx": idx, "w": w, "scores": s, "logits_grad": _exact_route_grad(st, idx, s, case["norm"], case["score"])}
    if op == "quantize":
        if case["kind"] == "rows":
            return _exact_rows(st["x"])
        v = _exact_matrix(st["x"])
        return {"values": v, "transposed": v.transpose(1, 2).contiguous()}
    if op in ("matmul", "swiglu"):
        at = torch.arange(case["k"], device="cuda") // BLOCK
        a = _exact_decode(st["a"]) * st["a_s"].double()[:, at]
        return (_exact_product if op == "matmul" else _exact_swiglu)(a, st["w"], st["offsets"])
    if op == "backward":
        grad, x, ends = st["grad"].double(), st["x"].double(), st["offsets"].tolist()
        dw = torch.zeros(case["experts"], case["n"], case["k"], dtype=torch.float64, device="cuda")
        for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if hi > lo:
                dw[e] = _exact_rows(grad[lo:hi].t().contiguous()) @ _exact_rows(x[lo:hi].t().contiguous()).t().contiguous()
        return {"x_grad": _exact_product(_exact_rows(grad), st["wt"], st["offsets"]), "w_grad": dw}
    idx, w, _ = _exact_route(st["logits"], st["bias"], case["top"], "sigmoid", case["groups"], case["kept"], True)
    x = _exact_rows(st["x"])
    pairs = sorted((e, a) for a, e in enumerate(idx.reshape(-1).tolist()))
    ends = [0] * (case["experts"] + 1)
    for e, _ in pairs:
        ends[e + 1] += 1
    offsets = torch.tensor(ends).cumsum(0).cuda()
    order = torch.tensor([a for _, a in pairs]).cuda()
    h = _exact_rows(_exact_swiglu(x[order // case["top"]], st["gate_up"], offsets))
    rows = torch.empty(order.numel(), case["hidden"], dtype=torch.float64, device="cuda")
    rows[order] = _exact_product(h, st["down"], offsets)
    return {"idx": idx, "y": (w.unsqueeze(2) * rows.unflatten(0, idx.shape)).sum(1)}
