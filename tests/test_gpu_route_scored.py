"""GPU tests of the router by scores (binade_moe_route_scored) and its backward
against their formulas in 64 bits.

Choices, counts and flags have to be equal. u = 2^-24, D the spread of a row's
logits. A score (relative to the row's largest) is an exponential of a rounded
difference, off by (2 D + 4) u, over 1 + an exponential, a Newton inverse and a
product: within (2 D + 12) u; a weight is one over a sum of up to 64 of them
(6 levels of a tree and the lanes' own 16), times scale: within
(4 D + 64) u relative. A gradient is such a quotient times a difference of two
numbers that each err relative to their largest term: within (8 D + 128) u of
the quotient times the terms' magnitudes."""
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


def make(T, E, seed, dtype, closed=0, coarse=False):
    g = gen(seed)
    x = torch.randn(T, E, generator=g) * 2
    if coarse:
        x = x.round()
    if closed:
        x[:, torch.randperm(E, generator=g)[:closed]] = -INF
    return x.to(dtype)


def ref_scores(x, score):
    x = x.double()
    return torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)


def ref_choice(x, k, score="softmax", bias=None, groups=1, top_groups=1, best=2):
    """Python lists of each row's experts, row by row."""
    s = ref_scores(x, score)
    v = s if bias is None else s + bias.double()
    # without bias the order is the logits': scores that round to one number differ
    key = x.double() if bias is None else v
    out = []
    for t in range(x.shape[0]):
        fine = [e for e in range(x.shape[1]) if x[t, e] > -INF and float(v[t, e]) > -INF]
        if groups > 1:
            size = x.shape[1] // groups
            score_of = {}
            for g in range(groups):
                src = key if bias is None and best == 1 else v
                mine = sorted((float(src[t, e]) for e in fine if e // size == g), reverse=True)[:best]
                if mine:
                    score_of[g] = sum(mine)
            keep = set(sorted(score_of, key=lambda g: (-score_of[g], g))[:top_groups])
            fine = [e for e in fine if e // size in keep]
        out.append(sorted(fine, key=lambda e: (-float(key[t, e]), e))[:k])
    return out


def ref_route(x, k, renorm=True, scale=1.0, valid=None, **rule):
    T, E = x.shape
    s = ref_scores(x, rule.get("score", "softmax"))
    q = s / s.sum(1, keepdim=True)
    idx = torch.full((T, k), -1, dtype=torch.int64)
    w = torch.zeros(T, k, dtype=torch.float64)
    counted = torch.zeros(T, dtype=torch.bool)
    for t, e in enumerate(ref_choice(x, k, **rule)):
        if (valid is not None and not valid[t]) or not e:
            continue
        counted[t] = True
        idx[t, :len(e)] = torch.tensor(e)
        w[t, :len(e)] = scale * s[t, e] / (s[t, e].sum() if renorm else 1.0)
    counts = torch.bincount(idx.flatten() + 1, minlength=E + 1)[1:]
    rows = int(counted.sum())
    ps = q[counted].sum(0)
    n = max(rows, 1)
    loss = E * float((counts.double() / (k * n) * (ps / n)).sum())
    return idx, w, torch.cat([counts, torch.tensor([rows])]), ps, loss


def check(x, k, r, renorm, scale, valid=None, stats=True, **rule):
    idx, w, counts, ps, loss = ref_route(x, k, renorm, scale, valid, **rule)
    assert torch.equal(r.idx.cpu().long(), idx)
    fin = torch.where(x > -INF, x, 0.0).double()
    D = float((fin.amax(1) - fin.amin(1)).max()) + float(fin.abs().max())
    tol = (4 * D + 64) * U
    assert torch.all((r.weights.cpu().double() - w).abs() <= tol * w.abs() + 1e-37)
    if not stats:
        assert r.counts is None and r.loss is None
        return
    assert torch.equal(r.counts.cpu().long(), counts)
    assert torch.all((r.prob_sum.cpu().double() - ps).abs() <= (tol + 64 * U) * ps + 1e-37)
    assert abs(float(r.loss) - loss) <= (tol + 64 * U) * loss + 1e-37


CASES = [  # T, E, k, groups, top_groups, best
    (1, 256, 8, 8, 4, 2), (1, 1, 1, 1, 1, 2), (33, 60, 4, 6, 2, 2), (200, 160, 6, 8, 3, 1), (67, 64, 8, 64, 9, 2),
    (40, 128, 16, 4, 2, 2), (9, 512, 64, 2, 1, 1), (21, 1024, 10, 32, 5, 2), (130, 7, 3, 7, 4, 2),
    (65, 65, 5, 5, 2, 1), (300, 300, 1, 3, 1, 2), (50, 8, 2, 1, 1, 2), (12, 1000, 8, 8, 8, 2),
    (17, 2, 2, 2, 2, 1), (500, 96, 8, 4, 1, 2)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,top_groups,best", CASES)
def test_route(T, E, k, groups, top_groups, best, score, dtype):
    say("route", T, E, k, groups, top_groups, best, score, dtype)
    x = make(T, E, T + E, dtype)
    bias = torch.randn(E, generator=gen(1)) * 0.2
    for b, renorm, scale in ((bias, True, 2.5), (None, False, 1.5), (torch.zeros(E), True, 1.0),
                             (None, True, 0.5)):
        rule = dict(score=score, groups=groups, top_groups=top_groups)
        r = B.moe_route(x.to(DEV), k, renormalize=renorm, bias=None if b is None else b.to(DEV),
                        group_best=best, scale=scale, **rule)
        check(x, k, r, renorm, scale, bias=b, best=best, **rule)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_ties_padding_and_closed(score):
    """Coarse logits tie all over, with every kind of bias; closed experts leave
    slots and whole groups empty, padded rows have none."""
    g = gen(2)
    for T, E, k, groups, top, best in ((64, 32, 8, 4, 2, 2), (70, 256, 8, 8, 4, 2), (40, 96, 12, 3, 1, 1)):
        for closed in (0, E // 2, E - 3, E):
            x = make(T, E, closed + E, BF, closed, coarse=True)
            valid = torch.rand(T, generator=g) < 0.7
            for b in (None, torch.zeros(E), torch.full((E,), 0.25), (torch.rand(E, generator=g) * 4).round() / 4):
                rule = dict(score=score, groups=groups, top_groups=top)
                r = B.moe_route(x.to(DEV), k, bias=None if b is None else b.to(DEV), valid=valid.to(DEV),
                                group_best=best, **rule)
                check(x, k, r, True, 1.0, valid, bias=b, best=best, **rule)


def test_route_near_ties_go_by_64_bits():
    """Values that differ by less than fp32 resolves: score + bias of neighbours
    are within 2^-30, so rows have to be settled in 64 bits."""
    E, T = 64, 48
    g = gen(3)
    x = torch.randn(T, E, generator=g)
    target = 0.5
    bias = torch.empty(E)
    base = torch.randn(E, generator=g)
    s = torch.sigmoid(base.double())
    bias = (target - s).float()                     # base row: all values within 2^-25 of target
    x = base[None, :].repeat(T, 1)
    x = x + torch.randint(-1, 2, (T, E), generator=g) * 2.0 ** -22
    r = B.moe_route(x.to(DEV), 8, score="sigmoid", bias=bias.to(DEV), groups=4, top_groups=2)
    check(x, 8, r, True, 1.0, score="sigmoid", bias=bias, groups=4, top_groups=2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_far_logits(score):
    """Scores far below what fp32 holds keep their quotients; a bias takes
    experts that score hundreds below the best."""
    g = gen(4)
    x = torch.randn(30, 64, generator=g) - 200.0
    r = B.moe_route(x.to(DEV), 6, score=score, bias=torch.zeros(64, device=DEV), groups=2)
    s = x.double().exp() if score == "sigmoid" else torch.softmax(x.double(), 1)
    # scores of 1e-87: their 64-bit values order them, the quotients are exp's
    idx, w, *_ = ref_route(x, 6, score=score, bias=torch.zeros(64), groups=2, top_groups=1)
    assert torch.equal(r.idx.cpu().long(), idx)
    assert torch.all((r.weights.cpu().double() - w).abs() <= (4 * 210 + 64) * U * w)
    # the bias decides
    x = torch.randn(20, 64, generator=g)
    x[:, :8] -= 150.0
    bias = torch.zeros(64)
    bias[:8] = torch.arange(8) + 5.0
    for k in (3, 8, 10):
        r = B.moe_route(x.to(DEV), k, score=score, bias=bias.to(DEV), stats=False)
        idx, w, *_ = ref_route(x, k, score=score, bias=bias)
        assert torch.equal(r.idx.cpu().long(), idx)
        assert torch.all((r.weights.cpu().double() - w).abs() <= (4 * 320 + 64) * U * w + 1e-37)
        d = B.moe_route_grad(x.to(DEV), r.idx, dweights=torch.ones(20, k, device=DEV), score=score,
                             bias=bias.to(DEV))
        assert torch.isfinite(d).all()
    del s


def test_route_special_values():
    E, k = 32, 4
    x = make(6, E, 5, F32)
    x[0, 3] = math.nan
    x[1, 7] = INF
    x[2, :] = -INF
    x[3, :] = math.nan
    x[4, 1:] = -INF
    bias = torch.zeros(E)
    bias[5], bias[6], bias[9] = INF, -INF, math.nan
    r = B.moe_route(x.to(DEV), k, score="sigmoid", bias=bias.to(DEV), stats=False)
    idx, w = r.idx.cpu(), r.weights.cpu()
    for t in (0, 1, 5):
        assert idx[t, 0] == 5 and not {6, 9} & set(idx[t].tolist()), idx[t]
        assert torch.isfinite(w[t]).all()
    assert 3 not in idx[0].tolist()
    assert (idx[2] == -1).all() and (idx[3] == -1).all() and not w[2].any() and not w[3].any()
    assert idx[4].tolist() == [0, -1, -1, -1] and w[4].tolist() == [1.0, 0.0, 0.0, 0.0]
    r = B.moe_route(x.to(DEV), k, score="softmax", bias=torch.zeros(E, device=DEV), stats=False)
    idx, w = r.idx.cpu(), r.weights.cpu()
    assert w[0].isnan().all() and w[1].isnan().all() and (idx[0] >= 0).all() and idx[1, 0] == 7
    assert 3 not in idx[0].tolist()


def ref_grad(x, idx, dw, counts, dloss, renorm, score, scale):
    """(gradient, terms' magnitudes) in 64 bits."""
    x, dw = x.double(), dw.double()
    T, E = x.shape
    k = idx.shape[1]
    s = ref_scores(x, score)
    rest = 1 - s if score == "sigmoid" else torch.ones_like(s)
    if score == "sigmoid":
        rest = torch.sigmoid(-x)
    at, keep = idx.clamp(min=0).long(), (idx >= 0).double()
    u = torch.zeros_like(s).scatter_add_(1, at, dw * keep)
    h = torch.zeros_like(s).scatter_add_(1, at, keep)
    if renorm:
        t = s / (s * h).sum(1, keepdim=True)
        t = torch.where(h > 0, t, 0.0)
        mean = (t * u).sum(1, keepdim=True)
        d = scale * t * (u - h * mean)
        big = scale * t * (u.abs() + h * (t * u.abs()).sum(1, keepdim=True))
    elif score == "sigmoid":
        d, big = scale * s * u, scale * s * u.abs()
    else:
        d = scale * s * (u - (s * u).sum(1, keepdim=True))
        big = scale * s * (u.abs() + (s * u.abs()).sum(1, keepdim=True))
    if counts is not None:
        rows = max(int(counts[E]), 1)
        f = dloss * E * counts[:E].double() / (k * rows * rows)
        q = s / s.sum(1, keepdim=True)
        d = d + q * (f - (q * f).sum(1, keepdim=True))
        big = big + q * (f.abs() + (q * f.abs()).sum(1, keepdim=True))
    on = (idx[:, :1] >= 0)
    return torch.where(on, d * rest, 0.0), torch.where(on, big * rest, 0.0)


@pytest.mark.parametrize("dtype,out", [(BF, F32), (F32, F32), (BF, BF), (F32, BF)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (333, 60, 4), (100, 300, 9), (21, 1024, 16), (64, 2, 1), (40, 128, 64)])
def test_grad(T, E, k, score, dtype, out):
    say("grad", T, E, k, score, dtype, out)
    g = gen(T)
    x = make(T, E, T * 3 + E, dtype)
    x[0, 0] = -INF
    bias = torch.randn(E, generator=g) * 0.3
    dw = torch.randn(T, k, generator=g)
    valid = torch.rand(T, generator=g) < 0.8
    for renorm in (True, False):
        r = B.moe_route(x.to(DEV), k, renormalize=renorm, score=score, bias=bias.to(DEV), scale=1.75,
                        valid=valid.to(DEV))
        idx = r.idx.cpu()
        for balance in (True, False):
            counts = r.counts.cpu() if balance else None
            d = B.moe_route_grad(x.to(DEV), r.idx, dweights=dw.to(DEV), counts=r.counts if balance else None,
                                 dloss=torch.full((1,), 0.5, device=DEV) if balance else None,
                                 renormalize=renorm, score=score, bias=bias.to(DEV), scale=1.75,
                                 out_dtype=out).cpu().double()
            ref, big = ref_grad(x, idx, dw, counts, 0.5, renorm, score, 1.75)
            fin = torch.where(x > -INF, x, 0.0).double()
            D = (fin.amax(1, keepdim=True) - fin.amin(1, keepdim=True)) + fin.abs().amax(1, keepdim=True)
            tol = (8 * D + 128) * U * big + (2.0 ** -8 * ref.abs() if out == BF else 0.0) + 1e-38
            assert torch.all((d - ref).abs() <= tol), (renorm, balance, ((d - ref).abs() / tol).max())


def test_grad_against_differences():
    """Central differences of the forward call's own weights and loss, in the
    logits, at fixed choices: h = 2^-7, whose square times a third derivative
    (below 8 here) and fp32's rounding over h stay under 2e-3 of the terms."""
    E, k = 24, 4
    g = gen(8)
    x = torch.randn(1, E, generator=g)
    bias = torch.randn(E, generator=g)
    dw, dl, h = torch.randn(1, k, generator=g), 0.7, 2.0 ** -7
    for score in ("sigmoid", "softmax"):
        for renorm in (True, False):
            kw = dict(renormalize=renorm, score=score, bias=bias.to(DEV), groups=4, top_groups=2, scale=1.5)
            r = B.moe_route(x.to(DEV), k, **kw)
            d = B.moe_route_grad(x.to(DEV), r.idx, dweights=dw.to(DEV), counts=r.counts,
                                 dloss=torch.full((1,), dl, device=DEV), renormalize=renorm, score=score,
                                 bias=bias.to(DEV), scale=1.5).cpu()[0]

            def value(y):
                q = B.moe_route(y.to(DEV), k, **kw)
                assert torch.equal(q.idx, r.idx)
                return float((q.weights.cpu().double() * dw.double()).sum()) + dl * float(q.loss)

            for e in range(E):
                up, down = x.clone(), x.clone()
                up[0, e] += h
                down[0, e] -= h
                num = (value(up) - value(down)) / float(up[0, e] - down[0, e])
                assert abs(num - float(d[e])) <= 2e-3 * (1 + float(dw.abs().sum())), (score, renorm, e)


def test_defaults_are_the_plain_router():
    """Without a rule nothing changes: the same bits as before."""
    x = make(500, 128, 1, BF).to(DEV)
    a, b = B.moe_route(x, 8), B.moe_route(x, 8, score="softmax", groups=1, scale=1.0)
    assert torch.equal(a.idx, b.idx) and torch.equal(a.weights, b.weights) and torch.equal(a.loss, b.loss)


def test_bad_index_strides_and_repeats():
    E, k, T = 40, 3, 50
    g = gen(6)
    wide = make(T, E + 9, 7, F32)
    x = wide[:, 3:E + 3]
    bias = torch.randn(E, generator=g)
    r = B.moe_route(wide.to(DEV)[:, 3:E + 3], k, score="sigmoid", bias=bias.to(DEV))
    check(x, k, r, True, 1.0, score="sigmoid", bias=bias)
    idx = r.idx.cpu().clone()
    idx[4] = torch.tensor([2, 2, 7])          # an expert twice
    idx[5, 1] = E                             # none of them
    idx[6, 2] = -3
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dw = torch.randn(T, k, generator=g)
    d = B.moe_route_grad(wide.to(DEV)[:, 3:E + 3], idx.to(DEV), dweights=dw.to(DEV), score="sigmoid",
                         scale=2.0, status=status).cpu().double()
    assert int(status) == B.DEV_BAD_INDEX
    idx[5, 1] = idx[6, 2] = -1
    ref, big = ref_grad(x, idx, dw, None, 0.0, True, "sigmoid", 2.0)
    assert torch.all((d - ref).abs() <= (8 * 16 + 128) * U * big + 1e-38)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_no_tokens(score):
    E = 24
    none = torch.empty(0, E, device=DEV)
    r = B.moe_route(none, 3, score=score, bias=torch.ones(E, device=DEV), groups=4, top_groups=2)
    assert r.idx.shape == (0, 3) and not bool(r.counts.any()) and not bool(r.prob_sum.any()) and float(r.loss) == 0
    d = B.moe_route_grad(none, r.idx, counts=r.counts, dloss=torch.ones(1, device=DEV), score=score, scale=2.0)
    assert d.shape == (0, E)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", [(700, 60, 4), (5000, 256, 8), (90, 1024, 20)])
def test_gradient_over_the_logits_themselves(T, E, k, score):
    x = make(T, E, 3, F32).to(DEV)
    r = B.moe_route(x, k, score=score, scale=1.5)
    dw, one = torch.randn(T, k, generator=gen(4)).to(DEV), torch.ones(1, device=DEV)
    args = dict(dweights=dw, counts=r.counts, dloss=one, score=score, scale=1.5)
    want = B.moe_route_grad(x, r.idx, **args)
    over = x.clone()
    assert B.moe_route_grad(over, r.idx, dlogits=over, **args) is over
    assert torch.equal(over, want)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,groups,top,best", [(64, 8, 8, 3, 2), (256, 8, 8, 4, 2), (60, 4, 6, 2, 1), (128, 12, 4, 2, 2),
                                                 (32, 4, 1, 1, 2)])
def test_special_biases_in_groups(E, k, groups, top, best, score):
    """A bias that is infinite or NaN: +inf comes first (equal ones, and groups
    that hold one, by rising number), -inf and NaN are never taken."""
    g = gen(11)
    for T, n_special in ((40, 1), (70, 5)):
        x = make(T, E, 12, F32)
        bias = torch.randn(E, generator=g) * 0.2
        at = torch.randperm(E, generator=g)
        bias[at[:n_special]] = INF
        bias[at[n_special:2 * n_special]] = -INF
        bias[at[2 * n_special:3 * n_special]] = math.nan
        bias[at[3 * n_special]] = -math.nan
        rule = dict(score=score, groups=groups, top_groups=top)
        r = B.moe_route(x.to(DEV), k, bias=bias.to(DEV), group_best=best, **rule)
        want = ref_choice(x, k, bias=bias, best=best, **rule)
        idx = r.idx.cpu().tolist()
        for t in range(T):
            assert idx[t] == want[t] + [-1] * (k - len(want[t])), (t, idx[t], want[t])
        assert torch.isfinite(r.weights).all()
        assert int(r.counts[:E].sum()) == sum(len(w) for w in want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,top_groups,best", [
    (513, 128, 6, 8, 3, 2), (600, 256, 8, 8, 4, 2), (520, 300, 10, 3, 2, 1), (700, 512, 8, 16, 4, 2),
    (515, 160, 16, 8, 3, 1), (1000, 65, 5, 5, 2, 2), (512, 512, 33, 8, 6, 2), (530, 96, 8, 1, 1, 2)])
def test_route_of_many_tokens(T, E, k, groups, top_groups, best, score, dtype):
    """From 513 tokens on a lane has sixteen experts instead of eight: rows that
    repeat, against the first ones by the formulas; plain values, and ties."""
    say("many", T, E, k, groups, top_groups, best, score, dtype)
    rows = 43
    times = -(-T // rows)
    valid = torch.rand(rows, generator=gen(2)) < 0.9
    coarse = (torch.rand(E, generator=gen(3)) * 4).round() / 4
    for b, ties in ((torch.randn(E, generator=gen(1)) * 0.2, False), (None, False), (coarse, True)):
        x = make(rows, E, T + E, dtype, closed=E // 9, coarse=ties)
        rule = dict(score=score, groups=groups, top_groups=top_groups)
        r = B.moe_route(x.repeat(times, 1).to(DEV), k, bias=None if b is None else b.to(DEV),
                        valid=valid.repeat(times).to(DEV), group_best=best, scale=2.5, **rule)
        idx, w, counts, ps, loss = ref_route(x, k, True, 2.5, valid, bias=b, best=best, **rule)
        assert torch.equal(r.idx.cpu().long(), idx.repeat(times, 1))
        fin = torch.where(x > -INF, x, 0.0).double()
        tol = (4 * (float((fin.amax(1) - fin.amin(1)).max()) + float(fin.abs().max())) + 64) * U
        assert torch.all((r.weights.cpu().double() - w.repeat(times, 1)).abs() <= tol * w.abs().repeat(times, 1) + 1e-37)
        assert torch.equal(r.counts.cpu().long(), counts * times)
        assert torch.all((r.prob_sum.cpu().double() - ps * times).abs() <= (tol + 64 * U) * ps * times + 1e-37)
        assert abs(float(r.loss) - loss) <= (tol + 64 * U) * loss + 1e-37


def test_near_ties_of_many_tokens():
    """Row by row the same choice as of few tokens, where neighbours' scores
    differ by less than fp32 resolves."""
    E, k = 256, 8
    base = torch.randn(90, 1, generator=gen(5)) + torch.randint(0, 40, (90, E), generator=gen(6)) * 2.0 ** -22
    x = base.to(DEV)
    bias = (torch.randint(0, 3, (E,), generator=gen(7)) * 2.0 ** -24).to(DEV)
    rule = dict(score="sigmoid", groups=8, top_groups=4)
    few = B.moe_route(x, k, bias=bias, **rule)
    many = B.moe_route(x.repeat(7, 1), k, bias=bias, **rule)
    assert torch.equal(many.idx.view(7, 90, k), few.idx.expand(7, 90, k))
    want = ref_choice(base, k, bias=bias.cpu(), best=2, **rule)
    assert few.idx.cpu().tolist() == want
