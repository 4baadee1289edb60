"""GPU tests of the router (binade_moe_route), its backward
(binade_moe_route_grad) and the combine's backward (binade_moe_combine_grad)
against their formulas in 64 bits.

Choices, counts and flags have to be equal. u = 2^-24. A weight is a
quotient of an exponential and a sum: exp of a difference d of fp32 logits is
off by 2 |d| u (the rounding of the difference and that of its product with
log2 e) and two steps for the function, the sum adds a tree of at most 16 + 6
levels, the quotients one step each: for |d| up to 26, which logits of the
scale drawn here (2) stay under, within 32 u + |d| u relative. Gradients subtract a mean:
they are held to their row's largest term, 64 u + |d| u of it."""
import ctypes
import math

import pytest
import torch

from decode_gemv_tensor_amd import binade as B

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
INF = math.inf


def say(*a):
    print(*a, flush=True)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def make_logits(T, E, seed, dtype, closed=0, coarse=False):
    g = gen(seed)
    x = torch.randn(T, E, generator=g) * 2
    if coarse:                         # many ties
        x = x.round()
    if closed:
        x[:, torch.randperm(E, generator=g)[:closed]] = -INF
    return x.to(dtype)


def ref_route(x, k, renorm, valid=None):
    """idx, weights (float64), counts, prob_sum, loss by the definition."""
    x = x.double()
    T, E = x.shape
    idx = torch.full((T, k), -1, dtype=torch.int64)
    w = torch.zeros(T, k, dtype=torch.float64)
    p = torch.softmax(x, 1)
    counted = torch.zeros(T, dtype=torch.bool)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    fine = (x > -INF).sum(1)
    for t in range(T):
        if valid is not None and not valid[t]:
            continue
        e = order[t, :min(k, int(fine[t]))]
        if not e.numel():
            continue
        counted[t] = True
        idx[t, :len(e)] = e
        w[t, :len(e)] = p[t, e] / (p[t, e].sum() if renorm else 1.0)
    counts = torch.bincount(idx.flatten() + 1, minlength=E + 1)[1:]
    counts = torch.cat([counts, counted.sum()[None]])
    rows = counts[E]
    ps = p[counted].sum(0)
    n = max(int(rows), 1)
    loss = E * float((counts[:E].double() / (k * n) * (ps / n)).sum())
    return idx, w, counts, ps, loss


CASES = [(1, 128, 8), (1, 1, 1), (4000, 256, 8), (3000, 513, 9), (3, 2, 2), (5, 60, 4), (16, 64, 6), (17, 65, 10), (33, 128, 8),
         (64, 256, 8), (67, 300, 1), (9, 512, 64), (21, 1024, 16), (1000, 16, 2), (5000, 8, 3),
         (130, 7, 7), (2100, 128, 8)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_route_against_the_definition(case, dtype):
    T, E, k = case
    g = gen(T + E)
    for renorm, closed, padded, coarse in [(True, 0, False, False), (False, E // 3, True, True),
                                           (True, E - 1, True, False)]:
        x = make_logits(T, E, T * E + k + closed, dtype, closed, coarse)
        valid = (torch.rand(T, generator=g) < 0.7) if padded else None
        idx, w, counts, ps, loss = ref_route(x, k, renorm, valid)
        say("route", case, dtype, renorm, closed, padded, coarse)
        v = None if valid is None else valid.to(DEV)
        r = B.moe_route(x.to(DEV), k, renormalize=renorm, valid=v)
        assert torch.equal(r.idx.cpu().long(), idx)
        assert torch.equal(r.counts.cpu().long(), counts)
        d = float((x.double().max(1, True).values - x.double()).nan_to_num(0, 0, 0).max())
        tol = (32 + min(d, 104)) * U
        assert bool(((r.weights.cpu().double() - w).abs() <= tol * w + 1e-37).all())
        # sums over the rows: per-lane chains of at most T / 4, then blocks
        chain = (math.sqrt(T) + 64) * U
        assert bool(((r.prob_sum.cpu().double() - ps).abs() <= (tol + chain) * ps + 1e-37).all())
        assert abs(float(r.loss) - loss) <= (tol + chain + 32 * U) * loss
        s = B.moe_route(x.to(DEV), k, renormalize=renorm, valid=v, stats=False)
        assert torch.equal(s.idx, r.idx) and torch.equal(s.weights, r.weights) and s.counts is None
        again = B.moe_route(x.to(DEV), k, renormalize=renorm, valid=v)
        assert torch.equal(again.prob_sum, r.prob_sum) and torch.equal(again.loss, r.loss)


def test_a_balanced_router_has_loss_one():
    E = 32
    x = torch.zeros(E, E)
    x[torch.arange(E), torch.arange(E)] = 3.0
    r = B.moe_route(x.to(DEV), 1)
    assert bool((r.counts[:E] == 1).all()) and int(r.counts[E]) == E
    assert abs(float(r.loss) - 1.0) <= 64 * U


def test_rows_without_an_expert_and_special_values():
    E, k = 20, 4
    x = make_logits(12, E, 3, F32)
    x[1] = -INF                                    # nothing to choose
    x[2] = -INF
    x[2, 7] = -3.0e38                              # one expert left, at the type's lowest
    x[3] = torch.finfo(F32).min                    # all equal at the lowest value
    x[4, 3] = float("nan")
    x[5, 6] = INF
    x[6, :] = float("nan")
    x[7, :] = 0.0
    x[7, 1::2] = -0.0                              # -0 and +0 tie
    x[8, 5], x[8, 9] = 200.0, 0.0                  # the others underflow
    r = B.moe_route(x.to(DEV), k)
    idx, w = r.idx.cpu(), r.weights.cpu()
    assert idx[1].tolist() == [-1] * k and not bool(w[1].any())
    assert idx[2].tolist() == [7, -1, -1, -1] and w[2].tolist() == [1.0, 0.0, 0.0, 0.0]
    assert idx[3].tolist() == [0, 1, 2, 3] and bool(((w[3] - 0.25).abs() <= 4 * U).all())
    assert 3 not in idx[4].tolist() and bool(torch.isnan(w[4]).all())
    assert idx[5, 0] == 6 and bool(torch.isnan(w[5]).any())
    assert idx[6].tolist() == [-1] * k
    assert idx[7].tolist() == [0, 1, 2, 3] and bool(((w[7] - 0.25).abs() <= 4 * U).all())
    assert idx[8, 0] == 5 and w[8, 0] == 1.0
    assert int(r.counts[E]) == 10 and bool(torch.isnan(r.loss).all())
    fine = x[[0, 2, 3, 7, 8, 9, 10, 11]]
    q = B.moe_route(fine.to(DEV), k)
    assert torch.equal(q.idx.cpu(), idx[[0, 2, 3, 7, 8, 9, 10, 11]])
    assert bool(torch.isfinite(q.loss).all())
    # the backward of rows without an expert is zero
    dw = torch.ones(12, k)
    d = B.moe_route_grad(x.to(DEV), r.idx, dweights=dw.to(DEV)).cpu()
    assert not bool(d[1].any()) and not bool(d[6].any())
    assert bool(torch.isfinite(d[[0, 2, 3, 7, 8, 9, 10, 11]]).all())


def test_no_tokens_and_all_padding():
    r = B.moe_route(torch.zeros(0, 16, device=DEV), 2)
    assert r.idx.shape == (0, 2) and not bool(r.counts.any()) and float(r.loss) == 0.0
    assert not bool(r.prob_sum.any())
    x = make_logits(9, 16, 1, BF).to(DEV)
    r = B.moe_route(x, 2, valid=torch.zeros(9, dtype=torch.bool, device=DEV))
    assert bool((r.idx == -1).all()) and not bool(r.weights.any()) and not bool(r.counts.any())
    assert float(r.loss) == 0.0
    d = B.moe_route_grad(x, r.idx, dweights=torch.ones(9, 2, device=DEV), counts=r.counts,
                         dloss=torch.ones(1, device=DEV))
    assert not bool(d.any())
    assert B.moe_route_grad(x[:0], r.idx[:0]).shape == (0, 16)


def ref_grad(x, idx, dw, counts, dloss, renorm):
    x = x.double()
    T, E = x.shape
    k = idx.shape[1]
    p = torch.softmax(x, 1)
    u = torch.zeros(T, E, dtype=torch.float64)
    if counts is not None:
        rows = max(int(counts[E]), 1)
        u += float(dloss) * E * counts[:E].double() / (k * rows * rows)
    terms = torch.zeros(T, 1, dtype=torch.float64)
    for t in range(T if dw is not None else 0):
        s = idx[t] >= 0
        if not bool(s.any()):
            continue
        e, g = idx[t, s].long(), dw[t, s].double()
        if renorm:
            total = p[t, e].sum()
            terms[t] = (g.abs().max() / total)
            g = (g - (g * p[t, e] / total).sum()) / total
        u[t].index_add_(0, e, g)
    d = p * (u - (p * u).sum(1, True))
    d[idx[:, 0] < 0] = 0
    scale = p * (u.abs().amax(1, True) + terms)
    return d, scale


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_route_grad_against_the_formula(case, dtype):
    T, E, k = case
    g = gen(T * 3 + E)
    for renorm, closed, padded in [(True, 0, False), (False, E // 3, True)]:
        x = make_logits(T, E, T + E + k, dtype, closed)
        valid = (torch.rand(T, generator=g) < 0.7).to(DEV) if padded else None
        r = B.moe_route(x.to(DEV), k, renormalize=renorm, valid=valid)
        dw = torch.randn(T, k, generator=g)
        dloss = torch.tensor([0.5])
        say("route_grad", case, dtype, renorm)
        diff = float((x.double().max(1, True).values - x.double()).nan_to_num(0, 0, 0).max())
        tol = (64 + min(diff, 104)) * U
        for w_, c_, l_ in [(dw, r.counts.cpu(), dloss), (dw, None, None),
                           (None, r.counts.cpu(), dloss)]:
            want, scale = ref_grad(x, r.idx.cpu(), w_, c_, l_, renorm)
            dev = lambda q: None if q is None else q.to(DEV)
            got = B.moe_route_grad(x.to(DEV), r.idx, dweights=dev(w_), counts=dev(c_),
                                   dloss=dev(l_), renormalize=renorm, out_dtype=F32)
            off = (got.cpu().double() - want).abs()
            assert bool((off <= tol * scale + 1e-37).all()), float((off - tol * scale).max())
            b = B.moe_route_grad(x.to(DEV), r.idx, dweights=dev(w_), counts=dev(c_),
                                 dloss=dev(l_), renormalize=renorm, out_dtype=BF)
            assert torch.equal(b, got.to(BF))


def test_route_grad_is_the_difference_of_the_forward():
    """Central differences of the kernel's own forward in fp32, step 2^-5: the
    third derivative of a softmax weight is below 1 and of the loss below its
    gradient's scale, so the difference is off by at most step^2 / 6 = 1.7e-4
    of dw's norm, and by 2 * 64 u / (2 step) = 1.2e-4 of it for rounding."""
    T, E, k = 24, 16, 3
    x = make_logits(T, E, 8, F32)
    for renorm in (True, False):
        r = B.moe_route(x.to(DEV), k, renormalize=renorm)
        g = gen(5)
        dw, dloss = torch.randn(T, k, generator=g), torch.tensor([3.0])
        grad = B.moe_route_grad(x.to(DEV), r.idx, dweights=dw.to(DEV), counts=r.counts,
                                dloss=dloss.to(DEV), renormalize=renorm).cpu().double()
        e = torch.randn(T, E, generator=g)
        e = e / e.abs().max()
        step = 2.0 ** -5
        order = torch.sort(x, 1, descending=True).values
        far = order[:, k - 1] - order[:, k] > 4 * step       # no choice changes on the way
        rows = far.nonzero()[:, 0]
        e[~far] = 0

        def f(sign):
            q = B.moe_route((x + sign * step * e).to(DEV), k, renormalize=renorm)
            assert torch.equal(q.counts, r.counts)
            at = {}
            for t in rows.tolist():
                at[t] = dict(zip(q.idx[t].tolist(), q.weights[t].tolist()))
            s = sum(float(dw[t, j]) * at[t][int(r.idx[t, j])] for t in rows.tolist()
                    for j in range(k))
            return s + 3.0 * float(q.loss)

        want = float((grad * e).sum())
        got = (f(1) - f(-1)) / (2 * step)
        norm = float(dw[rows].abs().sum()) + 3.0
        say("difference", got, want, norm)
        assert abs(got - want) <= 3e-4 * norm


def test_strides_duplicates_and_bad_indexes():
    T, E, k = 30, 24, 3
    x = make_logits(T, E, 2, F32)
    wide = torch.full((T, E + 7), 1e9)
    wide[:, :E] = x
    a, b = B.moe_route(x.to(DEV), k), B.moe_route(wide.to(DEV)[:, :E], k)
    assert torch.equal(a.idx, b.idx) and torch.equal(a.weights, b.weights)
    assert torch.equal(a.loss, b.loss)
    # the same index twice in a row adds both gradients; a bad one counts as none
    idx = a.idx.cpu().clone()
    idx[3] = torch.tensor([5, 5, 2])
    idx[4, 1] = E
    idx[5, 2] = -7
    dw = torch.randn(T, k, generator=gen(3))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = B.moe_route_grad(x.to(DEV), idx.to(DEV), dweights=dw.to(DEV), status=status)
    assert int(status.item()) == B.DEV_BAD_INDEX
    idx[4, 1] = idx[5, 2] = -1
    want, scale = ref_grad(x, idx, dw, None, None, True)
    assert bool(((got.cpu().double() - want).abs() <= 80 * U * scale + 1e-37).all())
    # through the C ABI: in place, and a strided output whose gaps stay
    d = x.to(DEV).clone()
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    args = (B._ptr(idx.to(DEV).contiguous()), B._ptr(dw.to(DEV)), None, None)
    keep = (idx.to(DEV).contiguous(), dw.to(DEV))
    args = (B._ptr(keep[0]), B._ptr(keep[1]), None, None)
    assert B.lib().binade_moe_route_grad(B._ptr(d), B.F32, E, T, E, k, 1, *args, B._ptr(d), B.F32,
                                         E, None, s) == B.OK
    out = torch.full((T + 1, E + 5), 9.0, device=DEV)
    xd = x.to(DEV)
    assert B.lib().binade_moe_route_grad(B._ptr(xd), B.F32, E, T, E, k, 1, *args, B._ptr(out),
                                         B.F32, E + 5, None, s) == B.OK
    torch.cuda.synchronize()
    assert torch.equal(d, got) and torch.equal(out[:T, :E], got)
    assert bool((out[T:] == 9).all()) and bool((out[:, E:] == 9).all())


@pytest.mark.parametrize("case", [(1, 1, 1), (1, 8, 2816), (3, 2, 7), (8, 8, 704), (5, 64, 33),
                                  (33, 10, 1001), (300, 3, 260), (2, 9, 5000)],
                         ids=lambda c: "x".join(map(str, c)))
def test_combine_grad(case):
    T, k, n = case
    g = gen(sum(case))
    y = torch.randn(T * k, n, generator=g)
    w = torch.rand(T, k, generator=g)
    for dt in (F32, BF):
        dout = torch.randn(T, n, generator=g).to(dt)
        dy_ref = w.reshape(T, k, 1).double() * dout.double().reshape(T, 1, n)
        prod = dout.double().reshape(T, 1, n) * y.double().reshape(T, k, n)
        dw_ref = prod.sum(2)
        for odt in (F32, BF):
            say("combine_grad", case, dt, odt)
            dy, dw = B.moe_combine_grad(y.to(DEV), w.to(DEV), dout.to(DEV), k, out_dtype=odt)
            # one fp32 product, rounded to the type
            assert torch.equal(dy.cpu(), (w.reshape(T, k, 1) * dout.float().reshape(T, 1, n))
                               .reshape(T * k, n).to(odt))
            # fma chains of n / 256 terms and a tree of 8 levels: n / 256 + 16 roundings
            tol = (n / 256 + 16) * U * prod.abs().sum(2)
            assert bool(((dw.cpu().double() - dw_ref).abs() <= tol).all())
            none, dw2 = B.moe_combine_grad(y.to(DEV), w.to(DEV).reshape(-1), dout.to(DEV), k,
                                           need_dy=False)
            assert none is None and torch.equal(dw2, dw.reshape(-1))
    assert rel_norm(dy_ref.reshape(T * k, n), dy.cpu()) <= 2.0 ** -8


def rel_norm(a, b):
    return float((a.double() - b.double()).norm() / max(float(a.double().norm()), 1e-300))


def test_combine_grad_without_columns_or_tokens():
    e = torch.empty(0, device=DEV)
    dy, dw = B.moe_combine_grad(e.reshape(6, 0), torch.ones(3, 2, device=DEV), e.reshape(3, 0), 2)
    assert dy.shape == (6, 0) and not bool(dw.any())
    dy, dw = B.moe_combine_grad(e.reshape(0, 5), e.reshape(0, 2), e.reshape(0, 5), 2)
    assert dy.shape == (0, 5) and dw.shape == (0, 2)


def test_many_tokens_of_many_slots():
    """Tokens enough for the kernel that shares dout among slots, slots beyond
    its eight, odd columns."""
    for T, k, n in ((600, 3, 37), (520, 11, 130)):
        g = gen(T)
        y = torch.randint(-4, 5, (T * k, n), generator=g).float()
        w = torch.randint(-3, 4, (T, k), generator=g).float()
        dout = torch.randint(-4, 5, (T, n), generator=g).float()
        dy, dw = B.moe_combine_grad(y.to(DEV), w.to(DEV), dout.to(DEV), k)
        assert torch.equal(dw.cpu(), (dout[:, None] * y.reshape(T, k, n)).sum(2))
        assert torch.equal(dy.cpu(), (w[:, :, None] * dout[:, None]).reshape(T * k, n))


@pytest.mark.parametrize("T,k,n", [((1 << 17) + 9, 3, 5), ((1 << 22) + 5, 8, 4)])
def test_more_tokens_than_one_axis_of_the_grid(T, k, n):
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    y = torch.randint(-4, 5, (T * k, n), generator=g, device=DEV).float()
    w = torch.randint(-3, 4, (T, k), generator=g, device=DEV).float()
    dout = torch.randint(-4, 5, (T, n), generator=g, device=DEV).float()
    dy, dw = B.moe_combine_grad(y, w, dout, k)
    assert torch.equal(dw, (dout[:, None] * y.reshape(T, k, n)).sum(2))
    assert torch.equal(dy, (w[:, :, None] * dout[:, None]).reshape(T * k, n))


def test_combine_grad_is_the_difference_of_the_combine():
    """moe_combine is linear in the weights and in y: exact on whole numbers."""
    T, k, n = 6, 4, 75
    g = gen(9)
    y = torch.randint(-5, 6, (T * k, n), generator=g).float().to(DEV)
    w = torch.randint(-3, 4, (T, k), generator=g).float().to(DEV)
    dout = torch.randint(-4, 5, (T, n), generator=g).float().to(DEV)
    dy, dw = B.moe_combine_grad(y, w, dout, k)
    f = lambda y_, w_: float((B.moe_combine(y_, w_.reshape(-1), k).double() * dout.double()).sum())
    ey = torch.randint(-1, 2, y.shape, generator=g).float().to(DEV)
    ew = torch.randint(-1, 2, w.shape, generator=g).float().to(DEV)
    assert f(y + ey, w) - f(y, w) == float((dy * ey).double().sum())
    assert f(y, w + ew) - f(y, w) == float((dw * ew).double().sum())


def test_streams_and_graphs():
    T, E, k, n = 70, 128, 8, 96
    g = gen(1)
    data = []
    for s in range(3):
        data.append({"x": make_logits(T, E, 40 + s, F32).to(DEV),
                     "valid": (torch.rand(T, generator=g) < 0.8).to(DEV),
                     "y": torch.randn(T * k, n, generator=g).to(DEV),
                     "dout": torch.randn(T, n, generator=g).to(DEV)})
    one = torch.ones(1, device=DEV)

    def go(d, stream=None):
        r = B.moe_route(d["x"], k, valid=d["valid"], stream=stream)
        dy, dw = B.moe_combine_grad(d["y"], r.weights, d["dout"], k, stream=stream)
        dx = B.moe_route_grad(d["x"], r.idx, dweights=dw, counts=r.counts, dloss=one,
                              stream=stream)
        return r.idx, r.weights, r.counts, r.prob_sum, r.loss, dy, dw, dx

    want = [go(d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [go(d, s) for d, s in zip(data, streams)]
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert all(torch.equal(i, j) for i, j in zip(p, q))
    buf = {key: t.clone() for key, t in data[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go(buf)
    for j in (1, 2, 0, 1, 2):
        for key, t in data[j].items():
            buf[key].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want[j]))
        go(data[j])                                # eager work between replays


def test_a_routed_layer_and_its_router_gradient():
    """Router -> gate and up experts -> SiLU * up -> down experts -> combine,
    then back to the logits, with packed experts, against float64 autograd
    over the same weights."""
    T, E, k, hid, ffn = 6, 8, 3, 64, 96
    g = gen(12)
    ws = [(torch.randn(E * n_, k_, generator=g) * 0.1).to(BF)
          for n_, k_ in ((ffn, hid), (ffn, hid), (hid, ffn))]
    r4 = [B.rice_to_r4(B.pack_rice(w).to(DEV)) for w in ws]
    x = torch.randn(T, hid, generator=g).to(BF)
    logits = make_logits(T, E, 77, F32)
    dout = torch.randn(T, hid, generator=g)
    r = B.moe_route(logits.to(DEV), k)
    gate = B.r4_moe_gemv(r4[0], E, x.to(DEV), r.idx)
    up = B.r4_moe_gemv(r4[1], E, x.to(DEV), r.idx)
    h = B.moe_silu_mul(gate, up)
    y = B.r4_moe_gemv(r4[2], E, h, r.idx, x_per_slot=True)
    out = B.moe_combine(y, r.weights.reshape(-1), k)
    _, dw = B.moe_combine_grad(y, r.weights, dout.to(DEV), k, need_dy=False)
    dloss = torch.full((1,), 0.01, device=DEV)
    grad = B.moe_route_grad(logits.to(DEV), r.idx, dweights=dw, counts=r.counts, dloss=dloss)

    q = logits.double().requires_grad_()
    p = torch.softmax(q, 1)
    idx = r.idx.cpu().long()
    pw = torch.gather(p, 1, idx)
    pw = pw / pw.sum(1, True)
    ye = torch.zeros(T, k, hid, dtype=torch.float64)
    we = [w.double().reshape(E, -1, w.shape[1]) for w in ws]
    for t in range(T):
        for s in range(k):
            e = int(idx[t, s])
            gt, u_ = we[0][e] @ x[t].double(), we[1][e] @ x[t].double()
            ye[t, s] = we[2][e] @ h[t * k + s].double().cpu()
            assert rel_norm(torch.nn.functional.silu(gt) * u_, h[t * k + s].cpu()) <= 2.0 ** -7
    ref = (pw[:, :, None] * ye).sum(1)
    assert rel_norm(ref.detach(), out.cpu()) <= 1e-5
    f = r.counts.cpu()[:E].double() / (k * T)
    loss = E * (f * p.mean(0)).sum()
    assert abs(float(loss.detach()) - float(r.loss)) <= 64 * U * float(loss.detach())
    ((ref * dout.double()).sum() + 0.01 * loss).backward()
    assert rel_norm(q.grad, grad.cpu()) <= 1e-5


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_a_workspace_of_the_size_asked_for_holds_it_all(dtype):
    """The caller's workspace, exactly as large as asked for, inside a larger
    buffer whose other bytes stay: on both sides of the step from four waves a
    block to sixteen, for every number of lanes a token."""
    for T, E, k in [(8192, 128, 8), (8193, 128, 8), (4096, 128, 8), (4000, 256, 8), (2049, 256, 8),
                    (2048, 512, 4), (1025, 512, 4), (1024, 1024, 8), (5, 1024, 64), (9000, 60, 2),
                    (0, 16, 2)]:
        say("workspace", T, E, k, dtype)
        x = make_logits(T, E, T + E, dtype).to(DEV)
        need = B.lib().binade_moe_route_workspace_bytes(T, E)
        pool = torch.full((2 * need + 512,), 0xFF, dtype=torch.uint8, device=DEV)
        assert pool.data_ptr() % 256 == 0
        got = B.moe_route(x, k, workspace=pool[256:256 + need])
        want = B.moe_route(x, k)
        assert bool((pool[:256] == 0xFF).all()) and bool((pool[256 + need:] == 0xFF).all())
        for name in ("idx", "weights", "counts", "prob_sum", "loss"):
            assert torch.equal(getattr(got, name), getattr(want, name)), name
        assert int(got.counts[E]) == T and int(got.counts[:E].sum()) == T * k
        with pytest.raises(B.BinadeError) as e:
            B.moe_route(x, k, workspace=pool[256:256 + need - 1])
        assert e.value.code == B.ENOSPACE


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_small_probabilities_do_not_lean_to_one_side(dtype):
    """Rows (0, -d) for d in 8..80, weights not renormalised: w1 is
    e / (1 + e) with e = exp(-d). The difference d is exact; its product with
    log2 e rounds by |d| u of e to either side, and what may lean to one side
    is at most the exponential's step (2 u), the sum (u), the reciprocal and
    the last product (u together, half steps either way): 4 u of w1. So every
    error is within (|d| + 8) u, and the mean of error / d is within 4 u times
    the mean of 1 / d, and four standard deviations of |d| u / sqrt(3) each."""
    g = gen(17)
    d = (8 + 72 * torch.rand(20000, generator=g)).to(dtype)
    x = torch.stack([torch.zeros_like(d), -d], 1)
    r = B.moe_route(x.to(DEV), 2, renormalize=False, stats=False)
    assert r.idx.cpu().tolist() == [[0, 1]] * d.numel()
    d = d.double()
    want = torch.exp(-d) / (1 + torch.exp(-d))
    off = (r.weights[:, 1].cpu().double() - want) / want
    say("leaning", float((off / d).mean()), float((off.abs() / ((d + 8) * U)).max()))
    assert bool((off.abs() <= (d + 8) * U).all())
    n = d.unique().numel()              # equal values err alike
    mean = float((off / d).mean())
    assert abs(mean) <= 4 * U * float((1 / d).mean()) + 4 * U / math.sqrt(3 * n)


def test_the_loss_is_that_of_its_counts_and_sums():
    """The summed probabilities are rounded once, for the output, and so is the
    loss, which comes from them unrounded: it is within u + u of the formula
    with the returned counts and sums."""
    for T, E, k, dtype in [(2048, 128, 8, F32), (8192, 128, 8, BF), (4000, 256, 8, BF),
                           (3000, 512, 4, F32), (60, 64, 6, F32), (700, 1000, 2, BF), (1, 8, 2, F32)]:
        for seed in range(4):
            x = make_logits(T, E, 100 * seed + E, dtype)
            r = B.moe_route(x.to(DEV), k)
            c, ps = r.counts.cpu().double(), r.prob_sum.cpu().double()
            want = E * float((c[:E] * ps).sum()) / (k * T * T)
            say("loss", T, E, (float(r.loss) - want) / want / U)
            assert abs(float(r.loss) - want) <= 2.01 * U * want
            assert int(c[E]) == T


def test_one_token_at_any_stride():
    E, k = 60, 4
    x = make_logits(1, E, 9, F32).to(DEV)
    want = B.moe_route(x, k)
    dw = torch.ones(1, k, device=DEV)
    grad = B.moe_route_grad(x, want.idx, dweights=dw, renormalize=False)
    for t in (x.reshape(E, 1).t(), x.as_strided((1, E), (3, 1))):
        got = B.moe_route(t, k)
        assert torch.equal(got.idx, want.idx) and torch.equal(got.weights, want.weights)
        assert torch.equal(B.moe_route_grad(t, want.idx, dweights=dw, renormalize=False), grad)
