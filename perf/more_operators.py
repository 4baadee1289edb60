"""What the 8-bit products and the router by scores of libbinade are measured on.

Two groups of operators of a mixture-of-experts model beside the packed
weights:

- matrix products in 8-bit floating point (e4m3) with a scale for each block
  of 128: of a projection (``f8_gemm``), its gradients (``f8_gemm_grad``) and
  of the experts that a router chose (``f8_moe_gemm``);
- the router by scores: sigmoid or softmax, a bias for balance, groups of
  experts, scaled weights (``moe_route`` with these arguments), and its
  gradient (``moe_route_grad``).

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is true, with this repository's kernels. Formulas:

  blocks     a block of 128 values v has the scale 2^e, e the least whole
             number >= -126 with max|v| <= 448 2^e (0 for a block of zeros),
             and the values Q(v) = 2^e e4m3(v 2^-e), to the nearest, ties to
             even; the last block of a row may be shorter
  product    y[t, n] = sum_k Q(x)[t, k] S[n / 128, k / 128] W[n, k], x in
             blocks along k, W e4m3 with one scale for 128 x 128 values
  gradients  dx[t, k] = sum_n Q(dy)[t, n] S W[n, k], dy in blocks along n;
             dw[n, k] = sum_t Q(dy)[t, n] Q(x)[t, k], both in blocks of 128
             rows t
  experts    y[t * top_k + s] = the product of x[t] with expert idx[t, s];
             zeros for -1
  router     s = sigmoid or softmax of the logits; v = s + bias, compared in
             64 bits; a group's score is the sum of its two best v (or the
             best one); only the top_groups best groups' experts can be
             taken; the top_k largest v of those, ties to the lowest expert,
             never an expert of logit -inf (such slots hold expert -1 and
             weight 0); w = s of the taken, over their sum if renormalised,
             times scale; counts, prob_sum P[e] = sum of s[e] / sum_j s[j]
             and the loss as moe_route has them
  backward   of sum(dw * w) + dloss * loss with respect to the logits
"""
import math

import torch

own = False

BF16, F32, E4M3, E8M0 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu
BYTES = {"bf16": 2, "f32": 4}
TYPES = {"bf16": BF16, "f32": F32}
BLOCK = 128


# ------------------------------------------------------------------- cases
def _gemm(name, m, n, k, scales, out):
    return {"name": name, "op": "f8_gemm", "m": m, "n": n, "k": k, "scales": scales, "out": out}


def _gemm_grad(name, m, n, k, scales, grads):
    return {"name": name, "op": "f8_gemm_grad", "m": m, "n": n, "k": k, "scales": scales,
            "grads": grads}


def _moe(name, tokens, experts, top_k, n, k, scales, padded, per_slot, out):
    return {"name": name, "op": "f8_moe_gemm", "tokens": tokens, "experts": experts,
            "top_k": top_k, "n": n, "k": k, "scales": scales, "padded": padded,
            "per_slot": per_slot, "out": out}


def _route(name, tokens, experts, top_k, logits, score, bias, groups, top_groups, best, renorm,
           scale, padded, closed, stats):
    return {"name": name, "op": "moe_route", "tokens": tokens, "experts": experts,
            "top_k": top_k, "logits": logits, "score": score, "bias": bias, "groups": groups,
            "top_groups": top_groups, "best": best, "renorm": renorm, "scale": scale,
            "padded": padded, "closed": closed, "stats": stats}


def _route_grad(name, *args):
    return _route(name, *args) | {"op": "moe_route_grad"}


def listed():
    return [
        # one request's token through the 12B up projection: latency and the
        # reading of the weights
        _gemm("product, one token", 1, 15360, 3840, "e8m0", "bf16"),
        # a decode step of 61 requests through the 12B down projection, from
        # a checkpoint whose scales are any fp32 numbers
        _gemm("product, decode batch", 61, 3840, 15360, "f32", "bf16"),
        # prompts of a dozen requests in one pass through the up projection
        _gemm("product, prompts", 4096, 15360, 3840, "e8m0", "bf16"),
        # a small ragged training batch with an odd output size, gradients in
        # the weights' type
        _gemm_grad("gradients, odd sizes", 2051, 1001, 2816, "f32", "bf16"),
        # a training step's backward through the up projection
        _gemm_grad("gradients, training step", 8192, 15360, 3840, "e8m0", "f32"),
        # gate products of the 128-expert layer for a step of 8 sequences
        _moe("experts, 8 tokens", 8, 128, 8, 704, 2816, "e8m0", False, False, "f32"),
        # its down products for a prompt batch with padded rows, each slot
        # with its own activations
        _moe("experts, prompts", 4096, 128, 8, 2816, 704, "f32", True, True, "bf16"),
        # the router of one decode token: sigmoid scores, balance bias, groups
        _route("router, one token", 1, 256, 8, "bf16", "sigmoid", True, 8, 4, 2, True, 2.5, False,
               0, False),
        # a training batch of it with its counts and balance loss
        _route("router, training batch", 65536, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5,
               False, 0, True),
        # softmax scores, the best expert a group, plain weights, padded rows
        # and closed experts of a prompt batch
        _route("router, prompts", 2049, 160, 6, "bf16", "softmax", False, 8, 3, 1, False, 16.0,
               True, 5, True),
        # a small batch's backward with an odd number of experts, no groups
        _route_grad("router backward, small", 333, 60, 4, "f32", "sigmoid", True, 1, 1, 2, False,
                    1.0, True, 0, True),
        # the training batch's backward
        _route_grad("router backward, training", 65536, 256, 8, "f32", "sigmoid", True, 8, 4, 2,
                    True, 2.5, False, 0, True),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    op = rng.choice(["f8_gemm", "f8_gemm", "f8_gemm_grad", "f8_gemm_grad", "f8_moe_gemm",
                     "f8_moe_gemm", "moe_route", "moe_route_grad"])
    scales, out = rng.choice(["e8m0", "f32"]), rng.choice(["bf16", "f32"])
    if op in ("f8_gemm", "f8_gemm_grad"):
        n, k = _spread(rng, 64, 15360), 32 * _spread(rng, 2, 480)
        if op == "f8_gemm":
            return _gemm("", _spread(rng, 1, 8192), n, k, scales, out)
        return _gemm_grad("", _spread(rng, 16, 8192), n, k, scales, out)
    if op == "f8_moe_gemm":
        experts = _spread(rng, 4, 256)
        return _moe("", _spread(rng, 1, 4096), experts, min(experts, rng.choice([1, 2, 4, 6, 8])),
                    _spread(rng, 64, 4096), 32 * _spread(rng, 2, 128), scales,
                    rng.random() < 0.5, rng.random() < 0.5, out)
    groups = rng.choice([1, 1, 2, 4, 8])
    experts = groups * _spread(rng, max(2, 8 // groups), 512 // groups)
    top_groups = rng.randint(1, groups)
    top_k = min(top_groups * (experts // groups), rng.choice([1, 2, 4, 6, 8, 10]))
    args = (_spread(rng, 1, 65536), experts, top_k, rng.choice(["bf16", "f32"]),
            rng.choice(["sigmoid", "softmax"]), rng.random() < 0.7, groups, top_groups,
            rng.choice([1, 2]), rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.random() < 0.5,
            rng.choice([0, 0, 1, experts // 3]), op == "moe_route_grad" or rng.random() < 0.7)
    return _route_grad("", *args) if op == "moe_route_grad" else _route("", *args)


def draw(rng):
    most = [work(c) for c in listed()]
    while True:
        c = _drawn(rng)
        w = work(c)
        if c["op"] == "f8_moe_gemm" and c["experts"] * c["n"] * c["k"] > 1 << 28:
            continue
        if c["op"].startswith("moe_route") and c["score"] == "softmax" and not c["bias"] and \
                c["groups"] == 1 and c["scale"] == 1.0:
            continue                # the plain softmax router is not this one
        if all(w[q] <= max(x[q] for x in most) for q in w):
            del c["name"]
            return c


def _blocks(n):
    return -(-n // BLOCK)


def _weight_bytes(c):
    """Of one matrix with its scales."""
    return c["n"] * c["k"] + _blocks(c["n"]) * _blocks(c["k"]) * (1 if c["scales"] == "e8m0" else 4)


def work(c):
    op = c["op"]
    if op == "f8_gemm":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": 2 * m * k + _weight_bytes(c) + m * n * BYTES[c["out"]],
                "flops": 2 * m * n * k}
    if op == "f8_gemm_grad":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": 2 * m * n + 2 * m * k + _weight_bytes(c) + 2 * m * k +
                n * k * BYTES[c["grads"]], "flops": 4 * m * n * k}
    t, e, s = c["tokens"], c["experts"], c["top_k"]
    if op == "f8_moe_gemm":
        rows = t * s if c["per_slot"] else t
        used = min(e, t * s)
        return {"bytes": 2 * rows * c["k"] + used * _weight_bytes(c) + 4 * t * s +
                t * s * c["n"] * BYTES[c["out"]], "flops": 2 * t * s * c["n"] * c["k"]}
    b = t * e * BYTES[c["logits"]] + 8 * t * s + (4 * e if c["bias"] else 0)
    if op == "moe_route":
        return {"bytes": b + (t if c["padded"] else 0) + (8 * e + 8 if c["stats"] else 0),
                "flops": 6 * t * e}
    return {"bytes": b + t * e * BYTES[c["logits"]] + 4 * e + 8, "flops": 10 * t * e}


# ------------------------------------------------------------------ inputs
def _quantised_weight(w, scales, g):
    """(e4m3 values, scales of 128 x 128 blocks) of fp32 w [..., n, k]."""
    n, k = w.shape[-2:]
    nb, kb = _blocks(n), _blocks(k)
    pad = torch.nn.functional.pad(w, (0, kb * BLOCK - k, 0, nb * BLOCK - n))
    tiles = pad.view(*w.shape[:-2], nb, BLOCK, kb, BLOCK)
    s = tiles.abs().amax((-3, -1)) / 448.0
    s = s * (1.0 + 2.0 ** -20)                    # nothing lands above 448
    if scales == "e8m0":
        s = _power(torch.ceil(torch.log2(s)))
    q = (tiles / s[..., :, None, :, None]).reshape(pad.shape)[..., :n, :k].to(E4M3).contiguous()
    return q, (s.to(E8M0) if scales == "e8m0" else s).contiguous()


def _valid(c, g):
    """Rows of four sequences, each padded behind its own length."""
    if not c["padded"]:
        return None
    t = c["tokens"]
    per = -(-t // 4)
    lens = torch.randint((per + 1) // 2, per + 1, (4,), generator=g, device="cuda")
    at = torch.arange(t, device="cuda")
    return at % per < lens[at // per]


def _like_activations(t, g):
    """Some columns are many times larger than the others, as a model's are."""
    big = torch.rand(t.shape[1], generator=g, device="cuda") < 0.01
    return t * torch.where(big, 16.0, 1.0)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, sigma=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=F32).mul_(sigma)

    s = {"case": c}
    if c["op"].startswith("f8"):
        shape = (c["n"], c["k"])
        if c["op"] == "f8_moe_gemm":
            t, e, kk = c["tokens"], c["experts"], c["top_k"]
            shape = (e, *shape)
            s["x"] = _like_activations(normal(t * kk if c["per_slot"] else t, c["k"]), g).to(BF16)
            # some experts are liked more than others
            liked = normal(t, e) + normal(e)
            s["idx"] = liked.topk(kk, dim=1).indices.to(torch.int32)
            valid = _valid(c, g)
            if valid is not None:
                s["idx"][~valid] = -1
        else:
            s["x"] = _like_activations(normal(c["m"], c["k"]), g).to(BF16)
        s["values"], s["scales"] = _quantised_weight(normal(*shape, sigma=c["k"] ** -0.5),
                                                     c["scales"], g)
        if c["op"] == "f8_gemm_grad":
            s["dy"] = (normal(c["m"], c["n"]) * torch.exp(normal(c["m"], 1)) * 1e-3).to(BF16)
        if own:
            from decode_gemv_tensor_amd import binade as B
            s["w"] = B.f8_weight(s["values"], s["scales"], train=c["op"] == "f8_gemm_grad")
        return s
    t, e = c["tokens"], c["experts"]
    logits = normal(t, e, sigma=1.5) + normal(e)
    if c["closed"]:
        logits[:, torch.randperm(e, generator=g, device="cuda")[:c["closed"]]] = -math.inf
    s["logits"] = logits.to(TYPES[c["logits"]])
    s["bias"] = normal(e, sigma=0.1) if c["bias"] else None
    s["valid"] = _valid(c, g)
    if c["op"] == "moe_route_grad":
        r = _route_plain(s)
        s["idx"], s["counts"] = r["idx"], r["counts"]
        s["dweights"] = normal(t, c["top_k"], sigma=1e-3)
        s["dloss"] = torch.full((1,), 1e-2, device="cuda")
    return s


# -------------------------------------------------------------- plain forms
def _power(e):
    """fp32 2^e of whole e in -126..127, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(F32)


def _q(v):
    """fp32 values of bf16 v quantised in blocks of 128 along the last axis."""
    n = v.shape[-1]
    pad = torch.nn.functional.pad(v.float(), (0, _blocks(n) * BLOCK - n))
    tiles = pad.view(*v.shape[:-1], -1, BLOCK)
    mant, ex = torch.frexp(tiles.abs().amax(-1, keepdim=True))
    e = torch.where(mant > 0, ex - 9 + (mant > 0.875).to(ex.dtype), 0).clamp(min=-126)
    back = (tiles * _power(-e)).to(E4M3).float() * _power(e)
    return back.view(pad.shape)[..., :n]


def _weight(values, scales):
    """fp32 [..., n, k] of e4m3 values and their blocks' scales."""
    n, k = values.shape[-2:]
    s = scales.float().repeat_interleave(BLOCK, -2)[..., :n, :]
    return values.float() * s.repeat_interleave(BLOCK, -1)[..., :k]


def _gemm_plain(s):
    return {"y": (_q(s["x"]) @ _weight(s["values"], s["scales"]).T).to(TYPES[s["case"]["out"]])}


def _gemm_grad_plain(s):
    dx = _q(s["dy"]) @ _weight(s["values"], s["scales"])
    dw = _q(s["dy"].T.contiguous()) @ _q(s["x"].T.contiguous()).T
    return {"dx": dx.to(BF16), "dw": dw.to(TYPES[s["case"]["grads"]])}


def _moe_plain(s):
    c = s["case"]
    x = _q(s["x"])
    idx = s["idx"].flatten().long()
    if not c["per_slot"]:
        x = x.repeat_interleave(c["top_k"], 0)
    if idx.numel() <= 64:
        e = idx.clamp(min=0)
        w = _weight(s["values"][e], s["scales"][e])
        y = torch.where(idx[:, None] >= 0, (w * x[:, None, :]).sum(2), 0.0)
        return {"y": y.to(TYPES[c["out"]])}
    y = torch.zeros(idx.numel(), c["n"], device=x.device)
    for e in range(c["experts"]):
        p = torch.nonzero(idx == e)[:, 0]
        y[p] = x[p] @ _weight(s["values"][e], s["scales"][e]).T
    return {"y": y.to(TYPES[c["out"]])}


def _scores(x, score):
    """Scores of logits in their own type (32 or 64 bits)."""
    if score == "softmax":
        p = torch.exp(x - x.max(1, keepdim=True).values)
        return p / p.sum(1, keepdim=True)
    e = torch.exp(-x.abs())
    return torch.where(x >= 0, 1.0, e) / (1.0 + e)


def _choice(x, bias, c):
    """(experts in falling order of their value, whether each can be taken)."""
    open_ = x > -math.inf
    v = _scores(x.double(), c["score"])
    if bias is not None:
        v = v + bias.double()
    v = torch.where(open_, v, -math.inf)
    if c["groups"] > 1:
        t, g = v.shape[0], c["groups"]
        best = torch.sort(v.view(t, g, -1), dim=2, descending=True).values[:, :, :c["best"]]
        some = best[:, :, 0] > -math.inf
        total = torch.where(best > -math.inf, best, 0.0).sum(2)
        at = torch.sort(torch.where(some, total, -math.inf), dim=1, descending=True,
                        stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros(t, g, dtype=torch.bool, device=v.device).scatter_(1, at, True)
        v = torch.where(keep.repeat_interleave(v.shape[1] // g, 1), v, -math.inf)
    v, at = torch.sort(v, dim=1, descending=True, stable=True)
    return at[:, :c["top_k"]], v[:, :c["top_k"]] > -math.inf


def _route_plain(s):
    c = s["case"]
    e, k = c["experts"], c["top_k"]
    x = s["logits"].float()
    at, keep = _choice(x, s["bias"], c)
    if s["valid"] is not None:
        keep = keep & s["valid"][:, None]
    row = keep[:, :1]
    sc = _scores(x, c["score"])
    w = torch.where(keep, torch.gather(sc, 1, at), 0.0)
    if c["renorm"]:
        w = torch.where(keep, w / w.sum(1, keepdim=True), 0.0)
    idx = torch.where(keep, at, -1).to(torch.int32)
    out = {"idx": idx, "weights": w * c["scale"]}
    if c["stats"]:
        rows = row.sum()
        chosen = torch.where(keep, at, e).flatten()
        counts = torch.zeros(e + 1, dtype=torch.int32, device=x.device)
        counts.scatter_add_(0, chosen, torch.ones_like(chosen, dtype=torch.int32))
        counts[e] = rows
        ps = torch.where(row, sc / sc.sum(1, keepdim=True), 0.0).sum(0)
        n = rows.clamp(min=1).float()
        out["counts"], out["prob_sum"] = counts, ps
        out["loss"] = (e * (counts[:e].float() / (k * n) * (ps / n)).sum()).reshape(1)
    return out


def _route_grad_plain(s):
    c = s["case"]
    e, k = c["experts"], c["top_k"]
    x, idx = s["logits"].float(), s["idx"].long()
    keep, at = idx >= 0, idx.clamp(min=0)
    sc = _scores(x, c["score"])
    dw = torch.where(keep, s["dweights"] * c["scale"], 0.0)
    if c["renorm"]:               # the slots' few values in 64 bits: they cancel
        taken = torch.where(keep, torch.gather(sc, 1, at), 0.0).double()
        total = taken.sum(1, keepdim=True)
        mean = (dw * (taken / total)).sum(1, keepdim=True)
        dw = torch.where(keep, (dw - mean) / total, 0.0).float()
    rows = s["counts"][e].clamp(min=1).float()
    f = s["dloss"] * e * s["counts"][:e].float() / (k * rows * rows)
    total = sc.sum(1, keepdim=True)
    ds = (f - (f * sc / total).sum(1, keepdim=True)) / total
    ds = ds.scatter_add(1, at, dw)
    if c["score"] == "softmax":
        d = sc * (ds - (sc * ds).sum(1, keepdim=True))
    else:
        d = sc * _scores(-x, "sigmoid") * ds
    return {"dlogits": torch.where(keep[:, :1], d, 0.0).to(TYPES[c["logits"]])}


PLAIN = {"f8_gemm": _gemm_plain, "f8_gemm_grad": _gemm_grad_plain, "f8_moe_gemm": _moe_plain,
         "moe_route": _route_plain, "moe_route_grad": _route_grad_plain}


# ------------------------------------------------------ the kernels' calls
def _own(s):
    from decode_gemv_tensor_amd import binade as B

    c = s["case"]
    if c["op"] == "f8_gemm":
        return {"y": B.f8_gemm(s["x"], s["w"], out_dtype=TYPES[c["out"]])}
    if c["op"] == "f8_gemm_grad":
        dx, dw = B.f8_gemm_grad(s["x"], s["w"], s["dy"], grad_dtype=TYPES[c["grads"]])
        return {"dx": dx, "dw": dw}
    if c["op"] == "f8_moe_gemm":
        return {"y": B.f8_moe_gemm(s["x"], s["w"], s["idx"], x_per_slot=c["per_slot"],
                                   out_dtype=TYPES[c["out"]])}
    if c["op"] == "moe_route":
        r = B.moe_route(s["logits"], c["top_k"], renormalize=c["renorm"], valid=s["valid"],
                        stats=c["stats"], score=c["score"], bias=s["bias"], groups=c["groups"],
                        top_groups=c["top_groups"], group_best=c["best"], scale=c["scale"])
        out = {"idx": r.idx, "weights": r.weights}
        return out | {"counts": r.counts, "prob_sum": r.prob_sum, "loss": r.loss} if c["stats"] \
            else out
    return {"dlogits": B.moe_route_grad(s["logits"], s["idx"], dweights=s["dweights"],
                                        counts=s["counts"], dloss=s["dloss"],
                                        renormalize=c["renorm"], out_dtype=TYPES[c["logits"]],
                                        score=c["score"], bias=s["bias"], groups=c["groups"],
                                        scale=c["scale"])}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------- 64-bit definitions
def _two_to(e):
    """fp64 2^e of whole e in -1000..1000, looked up."""
    table = torch.tensor([2.0 ** i for i in range(-1000, 1001)], dtype=torch.float64,
                         device=e.device)
    return table[e.long() + 1000]


def _log2_floor(v):
    """Whole exponent of positive v (fp64), exact at powers of two."""
    e = torch.floor(torch.log2(v))
    e = torch.where(_two_to(e) > v, e - 1, e)
    return torch.where(_two_to(e + 1) <= v, e + 1, e)


def _exact_q(v):
    """fp64 values of v [rows, n] rounded to e4m3 in blocks of 128 columns."""
    out = torch.empty(v.shape, dtype=torch.float64, device=v.device)
    for b in range(0, v.shape[1], BLOCK):
        part = v[:, b:b + BLOCK].double()
        top = part.abs().max(1, keepdim=True).values
        e = _log2_floor(top.clamp(min=1e-200)) - 8
        e = torch.where(top > 448.0 * _two_to(e), e + 1, e)
        e = torch.where(top == 0, torch.zeros_like(e), e.clamp(min=-126))
        u = part * _two_to(-e)
        step = _two_to(_log2_floor(u.abs().clamp(min=2.0 ** -6)) - 3)
        out[:, b:b + BLOCK] = torch.round(u / step) * step * _two_to(e)
    return out


def _exact_weight(values, scales):
    n, k = values.shape
    out = values.double()
    s = scales.double() if scales.dtype == F32 else scales.float().double()
    return out * s[(torch.arange(n, device=s.device) // BLOCK)[:, None],
                   (torch.arange(k, device=s.device) // BLOCK)[None, :]]


def _exact_route(s, c):
    e, k = c["experts"], c["top_k"]
    x = s["logits"].double()
    sc = torch.softmax(x, dim=1) if c["score"] == "softmax" else torch.special.expit(x)
    q = sc / sc.sum(1, keepdim=True)
    if c["op"] == "moe_route":
        shut = torch.isinf(x) & (x < 0)
        v = sc if s["bias"] is None else sc + s["bias"].double()[None, :]
        v = v.masked_fill(shut, -math.inf)
        if c["groups"] > 1:
            parts = v.reshape(-1, c["groups"], e // c["groups"])
            two = parts.topk(min(c["best"], parts.shape[2]), dim=2).values
            score = two.masked_fill(torch.isinf(two), 0.0).sum(2)
            score = score.masked_fill(torch.isinf(two).all(2), -math.inf)
            place = torch.argsort(torch.argsort(score, dim=1, descending=True, stable=True), dim=1)
            v = parts.masked_fill((place >= c["top_groups"])[:, :, None], -math.inf).reshape(v.shape)
        order = torch.argsort(v, dim=1, descending=True, stable=True)[:, :k]
        fine = ~torch.isinf(torch.gather(v, 1, order))
        if s["valid"] is not None:
            fine &= s["valid"][:, None]
        idx = order.masked_fill(~fine, -1)
        w = torch.gather(sc, 1, order) * fine
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        out = {"idx": idx.int(), "weights": w * c["scale"]}
        if not c["stats"]:
            return out
        counts = torch.bincount(idx.flatten() + 1, minlength=e + 1)[1:]
        live = fine.any(1)
        rows = int(live.sum())
        ps = q[live].sum(0)
        loss = e * float((counts.double() * ps).sum()) / (k * max(rows, 1) ** 2)
        out["counts"] = torch.cat([counts, counts.new_tensor([rows])]).int()
        out["prob_sum"] = ps
        out["loss"] = torch.tensor([loss], dtype=torch.float64, device=x.device)
        return out
    # d/dlogits by the chain rule: scores' Jacobian times what the weights and
    # the loss send back
    idx = s["idx"].long()
    rows = max(int(s["counts"][e]), 1)
    taken = torch.zeros_like(sc).scatter_add_(1, idx.clamp(min=0), (idx >= 0).double())
    up = torch.zeros_like(sc).scatter_add_(1, idx.clamp(min=0),
                                           s["dweights"].double() * (idx >= 0)) * c["scale"]
    if c["renorm"]:
        total = (sc * taken).sum(1, keepdim=True)
        up = taken * (up - (up * sc * taken).sum(1, keepdim=True) / total) / total
    load = float(s["dloss"]) * e * s["counts"][:e].double() / (k * rows * rows)
    up = up + (load[None, :] - q @ load[:, None]) / sc.sum(1, keepdim=True)
    if c["score"] == "softmax":
        d = sc * up - sc * (sc * up).sum(1, keepdim=True)
    else:
        d = sc * torch.special.expit(-x) * up
    return {"dlogits": torch.where(idx[:, :1] >= 0, d, torch.zeros_like(d))}


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] == "f8_gemm":
        return {"y": _exact_q(s["x"]) @ _exact_weight(s["values"], s["scales"]).T}
    if c["op"] == "f8_gemm_grad":
        dx = _exact_q(s["dy"]) @ _exact_weight(s["values"], s["scales"])
        dyt, xt = _exact_q(s["dy"].T), _exact_q(s["x"].T)
        return {"dx": dx, "dw": dyt @ xt.T}
    if c["op"] == "f8_moe_gemm":
        x, idx = _exact_q(s["x"]), s["idx"].flatten().long()
        y = torch.zeros(idx.numel(), c["n"], dtype=torch.float64, device=x.device)
        for e in range(c["experts"]):
            p = torch.nonzero(idx == e)[:, 0]
            rows = p if c["per_slot"] else torch.div(p, c["top_k"], rounding_mode="floor")
            y[p] = x[rows] @ _exact_weight(s["values"][e], s["scales"][e]).T
        return {"y": y}
    return _exact_route(s, c)
