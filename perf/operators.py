"""What the adapter and router operators of libbinade are measured on.

Two groups of operators stand beside the products of the packed weights:

- low-rank adapters of many requests beside one shared projection, forward
  (``lora_add``) and backward (``lora_grad``);
- the router around the expert products: choice of experts with per-expert
  counts and the balance loss (``moe_route``), its gradient
  (``moe_route_grad``), and the gradient of the weighted combine
  (``moe_combine_grad``) that gives the router its weights' gradient.

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is true, with this repository's kernels. Formulas:

  adapters   h[t] = A[id] x[t];  y[t] = base[t] + s[id] B[id] h[t]; rows with
             id < 0 have no adapter (h = 0, y = base)
  backward   g[t] = s[id] B[id]^T dy[t];  dx[t] = dx_base[t] + A[id]^T g[t];
             dA[a] = sum_{t: id = a} g[t] x[t]^T;
             dB[a] = sum_{t: id = a} s[a] dy[t] h[t]^T
  router     p = softmax(logits[t]); the top_k largest logits, ties to the
             lowest expert, never one of -inf (such slots hold expert -1 and
             weight 0); w = p of the chosen, over their sum if renormalised;
             counts[e] = slots that chose e, counts[E] = rows that count
             (valid ones with an expert); P[e] = sum of p over these rows;
             loss = E * sum_e counts[e] / (top_k rows) * P[e] / rows
  backward   of sum(dw * w) + dloss * loss with respect to the logits
  combine    out[t] = sum_s w[t, s] y[t, s]: dy[t, s] = w[t, s] dout[t],
             dw[t, s] = <dout[t], y[t, s]>
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
BYTES = {"bf16": 2, "f32": 4}
TYPES = {"bf16": BF16, "f32": F32}


# ------------------------------------------------------------------- cases
def _lora(name, m, n, k, rank, adapters, ids, base, out, keep):
    return {"name": name, "op": "lora_add", "m": m, "n": n, "k": k, "rank": rank,
            "adapters": adapters, "ids": ids, "base": base, "out": out, "keep": keep}


def _lora_grad(name, m, n, k, rank, adapters, ids, base, grads):
    return {"name": name, "op": "lora_grad", "m": m, "n": n, "k": k, "rank": rank,
            "adapters": adapters, "ids": ids, "base": base, "grads": grads}


def _route(name, tokens, experts, top_k, logits, renorm, padded, closed, stats):
    return {"name": name, "op": "moe_route", "tokens": tokens, "experts": experts,
            "top_k": top_k, "logits": logits, "renorm": renorm, "padded": padded,
            "closed": closed, "stats": stats}


def _route_grad(name, tokens, experts, top_k, logits, renorm, padded):
    return {"name": name, "op": "moe_route_grad", "tokens": tokens, "experts": experts,
            "top_k": top_k, "logits": logits, "renorm": renorm, "padded": padded, "closed": 0}


def _combine_grad(name, tokens, top_k, n, dout, out):
    return {"name": name, "op": "moe_combine_grad", "tokens": tokens, "top_k": top_k, "n": n,
            "dout": dout, "out": out}


def listed():
    return [
        # one request's token beside the 12B up projection: latency alone
        _lora("adapter, one token", 1, 15360, 3840, 16, 8, "row", "bf16", "bf16", False),
        # a decode step of 61 requests with 32 adapters beside the 12B down
        # projection, whose product arrives in fp32
        _lora("adapters, decode batch", 61, 3840, 15360, 32, 32, "row", "f32", "bf16", False),
        # prompts of a dozen requests in one pass (or a training forward over
        # several adapters, which keeps h) beside the 12B up projection
        _lora("adapters, prompts", 4096, 15360, 3840, 64, 16, "runs", "bf16", "bf16", True),
        # one adapter's training step beside the 12B up projection
        _lora_grad("adapter, training step", 8192, 15360, 3840, 16, 1, "one", "bf16", "f32"),
        # six tenants' adapters trained in one ragged batch, an odd output
        # size, gradients in the weights' type, nothing upstream to add to
        _lora_grad("adapters, six tenants", 2051, 1001, 2816, 64, 6, "runs", "none", "bf16"),
        # the router of one decode token of the 128-expert layer
        _route("router, one token", 1, 128, 8, "bf16", True, False, 0, False),
        # a prompt batch with padded rows and three closed experts
        _route("router, prompts", 2048, 128, 8, "f32", True, True, 3, True),
        # a training batch with its balance loss
        _route("router, training batch", 65536, 256, 8, "bf16", True, False, 0, True),
        # a small batch of an odd expert count, plain softmax weights
        _route_grad("router backward, small", 333, 60, 4, "f32", False, True),
        # the training batch's backward
        _route_grad("router backward, training", 65536, 256, 8, "bf16", True, False),
        # the combine's backward for the 8-token step of the 128-expert layer
        _combine_grad("combine backward, 8 tokens", 8, 8, 2816, "f32", "f32"),
        # and for a training batch of it
        _combine_grad("combine backward, training", 4096, 8, 2816, "bf16", "bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    op = rng.choice(["lora_add", "lora_add", "lora_grad", "lora_grad", "moe_route",
                     "moe_route_grad", "moe_combine_grad"])
    if op in ("lora_add", "lora_grad"):
        train = op == "lora_grad"
        m = _spread(rng, 16 if train else 1, 8192 if train else 4096)
        n = _spread(rng, 64, 15360)
        k = 32 * _spread(rng, 2, 480)
        rank = 8 * _spread(rng, 1, 16)
        adapters = _spread(rng, 1, max(1, min(64, 1024 // rank)))
        ids = "one" if adapters == 1 else rng.choice(["row", "runs"])
        if m > 512 and ids == "row":
            ids = "runs"           # rows of one prompt stand together
        if train:
            return _lora_grad("", m, n, k, rank, adapters, ids, rng.choice(["bf16", "none"]),
                              rng.choice(["bf16", "f32"]))
        return _lora("", m, n, k, rank, adapters, ids, rng.choice(["bf16", "f32"]),
                     rng.choice(["bf16", "f32"]), rng.random() < 0.5)
    tokens = _spread(rng, 1, 65536)
    if op == "moe_combine_grad":
        tokens = _spread(rng, 1, 4096)
        return _combine_grad("", tokens, rng.choice([1, 2, 4, 6, 8, 10]), _spread(rng, 64, 4096),
                             rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]))
    experts = _spread(rng, 4, 512)
    top_k = min(experts, rng.choice([1, 2, 4, 6, 8, 10]))
    args = (tokens, experts, top_k, rng.choice(["bf16", "f32"]), rng.random() < 0.7,
            rng.random() < 0.5)
    if op == "moe_route_grad":
        return _route_grad("", *args)
    return _route("", *args, rng.choice([0, 0, 1, experts // 3]), rng.random() < 0.7)


def draw(rng):
    most = [work(c) for c in listed()]
    while True:
        c = _drawn(rng)
        w = work(c)
        if all(w[q] <= max(x[q] for x in most) for q in w):
            del c["name"]
            return c


def work(c):
    op = c["op"]
    if op in ("lora_add", "lora_grad"):
        m, n, k, r = c["m"], c["n"], c["k"], c["rank"]
        used = min(m, c["adapters"])
        b = 2 * m * k + 2 * used * r * (n + k) + 4 * used + (0 if c["ids"] == "one" else 4 * m)
        if op == "lora_add":
            b += m * n * (BYTES[c["base"]] + BYTES[c["out"]]) + (4 * m * r if c["keep"] else 0)
            return {"bytes": b, "flops": 2 * m * r * (n + k)}
        b += 2 * m * n + 4 * m * r + m * k * (2 if c["base"] == "none" else 4)
        b += c["adapters"] * r * (n + k) * BYTES[c["grads"]]
        return {"bytes": b, "flops": 4 * m * r * (n + k)}
    if op == "moe_combine_grad":
        t, s, n = c["tokens"], c["top_k"], c["n"]
        return {"bytes": t * s * n * (4 + BYTES[c["out"]]) + t * n * BYTES[c["dout"]] + 8 * t * s,
                "flops": 3 * t * s * n}
    t, e, s = c["tokens"], c["experts"], c["top_k"]
    if op == "moe_route":
        b = t * e * BYTES[c["logits"]] + 8 * t * s + (t if c["padded"] else 0)
        return {"bytes": b + (8 * e + 8 if c["stats"] else 0), "flops": 4 * t * e}
    return {"bytes": 2 * t * e * BYTES[c["logits"]] + 8 * t * s + 4 * e + 8, "flops": 8 * t * e}


# ------------------------------------------------------------------ inputs
def _ids(c, g):
    m, a = c["m"], c["adapters"]
    if c["ids"] == "one":
        return None
    if c["ids"] == "row":          # each request its own adapter, some none
        return torch.randint(-1, a, (m,), generator=g, device="cuda").to(torch.int32)
    # ragged runs of rows of one request, about a dozen, some without adapter
    runs = max(1, min(12, m // 8))
    cuts = torch.randint(0, m, (runs - 1,), generator=g, device="cuda").sort().values
    run = torch.searchsorted(cuts, torch.arange(m, device="cuda"), right=True)
    return torch.randint(-1, a, (runs,), generator=g, device="cuda")[run].to(torch.int32)


def _valid(c, g):
    """Rows of four sequences, each padded behind its own length."""
    if not c["padded"]:
        return None
    t = c["tokens"]
    per = -(-t // 4)
    lens = torch.randint((per + 1) // 2, per + 1, (4,), generator=g, device="cuda")
    at = torch.arange(t, device="cuda")
    return at % per < lens[at // per]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=BF16, sigma=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=F32).mul_(sigma).to(dtype)

    s = {"case": c}
    if c["op"] in ("lora_add", "lora_grad"):
        m, n, k, r, na = c["m"], c["n"], c["k"], c["rank"], c["adapters"]
        s["x"] = normal(m, k)
        s["a"] = normal(na, r, k, sigma=k ** -0.5)
        s["b"] = normal(na, n, r, sigma=r ** -0.5)
        s["scale"] = torch.rand(na, generator=g, device="cuda") + 0.5
        s["ids"] = _ids(c, g)
        if c["op"] == "lora_add":
            s["base"] = normal(m, n, dtype=TYPES[c["base"]])
        else:
            s["dy"] = normal(m, n, sigma=1e-2)
            s["dx_base"] = None if c["base"] == "none" else normal(m, k, sigma=1e-2)
            s["h"] = _placed(s["x"].float() @ s["a"].float().flatten(0, 1).T, s, True)
        return s
    if c["op"] == "moe_combine_grad":
        t, kk, n = c["tokens"], c["top_k"], c["n"]
        s["y"] = normal(t * kk, n, dtype=F32)
        s["weights"] = torch.softmax(normal(t, kk, dtype=F32), 1).flatten()
        s["dout"] = normal(t, n, dtype=TYPES[c["dout"]], sigma=1e-2)
        return s
    t, e = c["tokens"], c["experts"]
    bias = normal(e, dtype=F32)    # some experts are liked more than others
    logits = normal(t, e, dtype=F32, sigma=1.5) + bias
    if c["closed"]:
        logits[:, torch.randperm(e, generator=g, device="cuda")[:c["closed"]]] = -math.inf
    s["logits"] = logits.to(TYPES[c["logits"]])
    s["valid"] = _valid(c, g)
    if c["op"] == "moe_route_grad":
        r = _route_plain(s)
        s["idx"], s["counts"] = r["idx"], r["counts"]
        s["dweights"] = normal(t, c["top_k"], dtype=F32, sigma=1e-3)
        s["dloss"] = torch.full((1,), 1e-2, device="cuda")
    return s


# -------------------------------------------------------------- plain forms
def _onehot(s):
    """fp32 [m, adapters]: 1 at each row's adapter."""
    na = s["case"]["adapters"]
    ids = s["ids"]
    if ids is None:
        return torch.ones(s["x"].shape[0], 1, device=s["x"].device)
    return (ids[:, None] == torch.arange(na, device=ids.device)).float()


def _placed(all_h, s, narrow):
    """[m, adapters * rank] products with every adapter -> each row's own
    block alone, in its place, or (narrow) as [m, rank]."""
    na, r = s["case"]["adapters"], s["case"]["rank"]
    own_block = all_h.view(-1, na, r) * _onehot(s)[:, :, None]
    return own_block.sum(1) if narrow else own_block.flatten(1)


def _lora_add_plain(s):
    c = s["case"]
    a, b = s["a"].float().flatten(0, 1), s["b"].float()
    h = _placed(s["x"].float() @ a.T, s, False)
    sb = (b * s["scale"][:, None, None]).transpose(1, 2).flatten(0, 1)     # [adapters*rank, n]
    y = (s["base"].float() + h @ sb).to(TYPES[c["out"]])
    if not c["keep"]:
        return {"y": y}
    return {"y": y, "h": h.view(c["m"], c["adapters"], c["rank"]).sum(1)}


def _lora_grad_plain(s):
    c = s["case"]
    na, r, t = c["adapters"], c["rank"], TYPES[c["grads"]]
    a, b, x, dy = s["a"].float().flatten(0, 1), s["b"].float(), s["x"].float(), s["dy"].float()
    sb = (b * s["scale"][:, None, None]).transpose(1, 2).flatten(0, 1)
    gp = _placed(dy @ sb.T, s, False)
    dx = gp @ a
    if s["dx_base"] is not None:
        dx = dx + s["dx_base"].float()
    hs = (s["h"][:, None, :] * (_onehot(s) * s["scale"])[:, :, None]).flatten(1)
    da = (gp.T @ x).view(na, r, -1)
    db = (dy.T @ hs).view(-1, na, r).transpose(0, 1)
    return {"dx": dx.to(BF16), "da": da.to(t), "db": db.to(t).contiguous()}


def _route_plain(s):
    c = s["case"]
    e, k = c["experts"], c["top_k"]
    x = s["logits"].float()
    row = (x > -math.inf).any(1)
    if s["valid"] is not None:
        row = row & s["valid"]
    order, at = torch.sort(x, dim=1, descending=True, stable=True)
    top = order[:, :k] > -math.inf
    keep = row[:, None] & top
    idx = torch.where(keep, at[:, :k], -1).to(torch.int32)
    p = torch.exp(x - order[:, :1])
    p = torch.where(row[:, None], p / p.sum(1, keepdim=True), 0.0)
    w = torch.where(keep, torch.gather(p, 1, at[:, :k]), 0.0)
    if c["renorm"]:
        w = torch.where(keep, w / w.sum(1, keepdim=True), 0.0)
    out = {"idx": idx, "weights": w}
    if c.get("stats", True):
        rows = row.sum()
        chosen = torch.where(keep, idx.long(), e).flatten()
        counts = torch.zeros(e + 1, dtype=torch.int32, device=x.device)
        counts.scatter_add_(0, chosen, torch.ones_like(chosen, dtype=torch.int32))
        counts[e] = rows
        ps = p.sum(0)
        n = rows.clamp(min=1).float()
        out["counts"], out["prob_sum"] = counts, ps
        out["loss"] = (e * (counts[:e].float() / (k * n) * (ps / n)).sum()).reshape(1)
    return out


def _route_grad_plain(s):
    c = s["case"]
    e, k = c["experts"], c["top_k"]
    x, idx = s["logits"].float(), s["idx"].long()
    row = idx[:, :1] >= 0
    keep = idx >= 0
    p = torch.exp(x - x.max(1, keepdim=True).values)
    p = p / p.sum(1, keepdim=True)
    dw = torch.where(keep, s["dweights"], 0.0)
    at = idx.clamp(min=0)
    if c["renorm"]:
        pc = torch.where(keep, torch.gather(p, 1, at), 0.0)
        total = pc.sum(1, keepdim=True)
        dw = torch.where(keep, (dw - (dw * pc / total).sum(1, keepdim=True)) / total, 0.0)
    rows = s["counts"][e].clamp(min=1).float()
    u = (s["dloss"] * e * s["counts"][:e].float() / (k * rows * rows)).expand_as(p)
    u = u.scatter_add(1, at, dw)
    d = p * (u - (p * u).sum(1, keepdim=True))
    return {"dlogits": torch.where(row, d, 0.0).to(TYPES[c["logits"]])}


def _combine_grad_plain(s):
    c = s["case"]
    t, k, n = c["tokens"], c["top_k"], c["n"]
    dout = s["dout"].float()
    dy = s["weights"].view(t, k, 1) * dout[:, None, :]
    dw = (dout[:, None, :] * s["y"].view(t, k, n)).sum(2)
    return {"dy": dy.view(t * k, n).to(TYPES[c["out"]]), "dweights": dw}


PLAIN = {"lora_add": _lora_add_plain, "lora_grad": _lora_grad_plain, "moe_route": _route_plain,
         "moe_route_grad": _route_grad_plain, "moe_combine_grad": _combine_grad_plain}


# ------------------------------------------------------ the kernels' calls
def _own(s):
    from decode_gemv_tensor_amd import binade as B

    c = s["case"]
    if c["op"] == "lora_add":
        got = B.lora_add(s["x"], s["a"], s["b"], s["ids"], base=s["base"], scale=s["scale"],
                         out_dtype=TYPES[c["out"]], keep_h=c["keep"])
        return {"y": got[0], "h": got[1]} if c["keep"] else {"y": got}
    if c["op"] == "lora_grad":
        dx, da, db = B.lora_grad(s["x"], s["a"], s["b"], s["ids"], s["dy"], h=s["h"],
                                 scale=s["scale"], dx_base=s["dx_base"],
                                 grad_dtype=TYPES[c["grads"]])
        return {"dx": dx, "da": da, "db": db}
    if c["op"] == "moe_route":
        r = B.moe_route(s["logits"], c["top_k"], renormalize=c["renorm"], valid=s["valid"],
                        stats=c["stats"])
        out = {"idx": r.idx, "weights": r.weights}
        return out | {"counts": r.counts, "prob_sum": r.prob_sum, "loss": r.loss} if c["stats"] \
            else out
    if c["op"] == "moe_route_grad":
        return {"dlogits": B.moe_route_grad(s["logits"], s["idx"], dweights=s["dweights"],
                                            counts=s["counts"], dloss=s["dloss"],
                                            renormalize=c["renorm"],
                                            out_dtype=TYPES[c["logits"]])}
    dy, dw = B.moe_combine_grad(s["y"], s["weights"], s["dout"], c["top_k"],
                                out_dtype=TYPES[c["out"]])
    return {"dy": dy, "dweights": dw.flatten().view(c["tokens"], c["top_k"])}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------- 64-bit definitions
def _exact_lora(s, c):
    m, n, k, r, na = c["m"], c["n"], c["k"], c["rank"], c["adapters"]
    dev = s["x"].device
    ids = torch.zeros(m, dtype=torch.int64, device=dev) if s["ids"] is None else s["ids"].long()
    x = s["x"].double()
    if c["op"] == "lora_add":
        y = s["base"].double()
        h = torch.zeros(m, r, dtype=torch.float64, device=dev)
        for a in range(na):
            t = torch.nonzero(ids == a)[:, 0]
            h[t] = x[t] @ s["a"][a].double().T
            y[t] += float(s["scale"][a]) * (h[t] @ s["b"][a].double().T)
        return {"y": y, "h": h} if c["keep"] else {"y": y}
    dy = s["dy"].double()
    dx = torch.zeros(m, k, dtype=torch.float64, device=dev)
    if s["dx_base"] is not None:
        dx += s["dx_base"].double()
    da = torch.zeros(na, r, k, dtype=torch.float64, device=dev)
    db = torch.zeros(na, n, r, dtype=torch.float64, device=dev)
    for a in range(na):
        t = torch.nonzero(ids == a)[:, 0]
        sc = float(s["scale"][a])
        grad = sc * (dy[t] @ s["b"][a].double())
        dx[t] += grad @ s["a"][a].double()
        da[a] = grad.T @ x[t]
        db[a] = sc * (dy[t].T @ s["h"][t].double())
    return {"dx": dx, "da": da, "db": db}


def _exact_route(s, c):
    e, k = c["experts"], c["top_k"]
    x = s["logits"].double()
    p = torch.softmax(x, dim=1)
    if c["op"] == "moe_route":
        live = torch.isfinite(x).any(1)
        if s["valid"] is not None:
            live &= s["valid"]
        # rank of each expert: how many are larger, or as large and before it
        order = torch.argsort(x, dim=1, descending=True, stable=True)[:, :k]
        fine = torch.isfinite(torch.gather(x, 1, order)) & live[:, None]
        idx = torch.where(fine, order, torch.full_like(order, -1))
        w = torch.gather(p, 1, order) * fine
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        out = {"idx": idx.int(), "weights": w}
        if not c["stats"]:
            return out
        counts = torch.bincount(idx.flatten() + 1, minlength=e + 1)[1:]
        rows = int(live.sum())
        ps = (p * live[:, None]).nan_to_num(0.0).sum(0)
        loss = e * float((counts.double() * ps).sum()) / (k * max(rows, 1) ** 2)
        out["counts"] = torch.cat([counts, counts.new_tensor([rows])]).int()
        out["prob_sum"] = ps
        out["loss"] = torch.tensor([loss], dtype=torch.float64, device=x.device)
        return out
    # d/dlogits of sum(dw * w) + dloss * loss through p's Jacobian
    idx = s["idx"].long()
    rows = max(int(s["counts"][e]), 1)
    up = torch.zeros_like(p) + float(s["dloss"]) * e * s["counts"][:e].double() / (k * rows * rows)
    chosen = torch.zeros_like(p)
    chosen.scatter_add_(1, idx.clamp(min=0), (idx >= 0).double())
    dw = torch.zeros_like(p)
    dw.scatter_add_(1, idx.clamp(min=0), s["dweights"].double() * (idx >= 0))
    if c["renorm"]:
        total = (p * chosen).sum(1, keepdim=True)
        w = p * chosen / total
        up = up + chosen * (dw - (dw * w).sum(1, keepdim=True)) / total
    else:
        up = up + dw
    d = p * up - p * (p * up).sum(1, keepdim=True)
    return {"dlogits": torch.where(idx[:, :1] >= 0, d, torch.zeros_like(d))}


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] in ("lora_add", "lora_grad"):
        return _exact_lora(s, c)
    if c["op"] == "moe_combine_grad":
        t, k, n = c["tokens"], c["top_k"], c["n"]
        dout, y = s["dout"].double(), s["y"].double().view(t, k, n)
        w = s["weights"].double().view(t, k)
        return {"dy": torch.einsum("ts,tn->tsn", w, dout).reshape(t * k, n),
                "dweights": torch.einsum("tn,tsn->ts", dout, y)}
    return _exact_route(s, c)
