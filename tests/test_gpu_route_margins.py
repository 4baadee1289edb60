"""GPU tests of choices that fp32 alone cannot make: the router by scores compares
score + bias in fp64, and a row may only be settled in fp32 where its gaps are
larger than everything that fp32 rounds. Inputs here bring gaps and roundings of
like size together; choices have to be those of 64 bits, row by row. (Exactly
equal values aside, the 64-bit values compared here are more than 2^-49 of the
larger apart, which fp64 resolves whichever way its sums are ordered: rows that
are nearer are left out, and have to be few.)"""
import math

import pytest
import torch

from decode_gemv_tensor_amd import binade as B

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
INF = math.inf


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def scores(x, score):
    x = x.double()
    return torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)


def choice(x, bias, k, score, groups=1, top_groups=1, best=2):
    """(experts [T, k], whether fp64 itself tells the row's values apart)."""
    T, E = x.shape
    v = scores(x, score) + bias.double()
    clear = torch.ones(T, dtype=torch.bool)

    def settle(values, size, n):          # n largest, ties to the lowest; are they clear?
        s, at = torch.sort(values, dim=1, descending=True, stable=True)
        m = min(n, values.shape[1] - 1)
        gap = s[:, :m] - s[:, 1:m + 1]
        return at[:, :n], ((gap == 0) | (gap > 2.0 ** -49 * size)).all(1)

    if groups > 1:
        part = torch.sort(v.view(T, groups, -1), dim=2, descending=True).values[:, :, :best]
        at, ok = settle(part.sum(2), part.abs().sum(2).amax(1, keepdim=True), top_groups)
        clear &= ok
        keep = torch.zeros(T, groups, dtype=torch.bool).scatter_(1, at, True)
        v = torch.where(keep.repeat_interleave(E // groups, 1), v, -INF)
    fin = torch.where(v > -INF, v, 0.0).abs().amax(1, keepdim=True)
    at, ok = settle(v, fin, k)
    return at, clear & ok


def agree(name, x, bias, k, few=0.02, **rule):
    want, clear = choice(x, bias, k, **rule)
    rule["group_best"] = rule.pop("best", 2)
    got = B.moe_route(x.to(DEV), k, bias=bias.to(DEV), stats=False, **rule).idx.cpu().long()
    wrong = ((got != want).any(1) & clear).sum().item()
    print(name, "wrong", wrong, "unclear", int((~clear).sum()), "of", len(x), flush=True)
    assert wrong == 0, name
    assert (~clear).float().mean() <= few


def test_a_group_whose_two_best_cancel():
    """Sums of 1.0197 and 1.0423 in 64 bits, 1.0625 and 1.0 in 32."""
    x = torch.tensor([[1.7583513, -1.6088977, -0.13181214, 0.30318862]])
    bias = torch.tensor([1e6, -1e6, 1e6, -1e6])
    assert choice(x, bias, 1, "sigmoid", 2, 1)[0].item() == 2
    agree("cancel", x, bias, 1, score="sigmoid", groups=2, top_groups=1)


# groups of whole lanes (8 and 16 experts a lane: more than 512 tokens) and others
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,groups,top_groups,k", [
    (500, 4, 2, 1, 1), (500, 64, 8, 3, 8), (4000, 256, 8, 4, 8), (500, 256, 8, 4, 12), (4000, 96, 8, 2, 4),
    (500, 60, 6, 2, 10), (4000, 512, 16, 4, 8), (400, 1024, 32, 5, 6)])
@pytest.mark.parametrize("size", [1.0, 20.0, 50.0, 1e3, 1e6, 1e30])
def test_large_biases_of_both_signs(T, E, groups, top_groups, k, score, size):
    """A group's best is far above nothing and its second best as far below."""
    g = gen(int(size) % 1000 + E)
    x = torch.randn(T, E, generator=g)
    near = x * 1e-3                                      # scores close together
    bias = torch.full((E,), -size)
    bias[torch.arange(groups) * (E // groups) + torch.randint(0, E // groups, (groups,), generator=g)] = size
    for name, rows in (("plain", x), ("near", near)):
        # at 1e30 scores do not move a sum of 64 bits: equal groups everywhere
        agree(name, rows, bias, k, 0.05 if size < 1e6 else 1.0, score=score, groups=groups, top_groups=top_groups)
        mixed = torch.where(torch.rand(E, generator=gen(3)) < 0.5, size, -size)
        agree(name + " mixed", rows, mixed, k, 1.0, score=score, groups=groups, top_groups=top_groups)


@pytest.mark.parametrize("T", [300, 3000])
@pytest.mark.parametrize("E", [64, 256, 1024])
def test_softmax_totals_that_lose_small_terms(T, E):
    """One expert near probability 1 beside many that fp32 drops one by one from
    the row's total, and another whose bias is as large as the first one's
    probability: gaps of 0 to 60 steps of 2^-24."""
    u = 2.0 ** -24
    for first in (0, E // 2 + 1):
        c = torch.linspace(0.80, 0.999, T)
        x = torch.full((T, E), 0.0)
        x += torch.log(c * u)[:, None]
        x[:, first] = 0.0
        for j in range(16):
            bias = torch.zeros(E)
            bias[E - 1] = 1.0 - (E - 1) * 0.9 * u + (j - 8) * 4 * u
            agree(f"total {first} {j}", x, bias, 1, score="softmax")
            agree(f"total {first} {j} in groups", x, bias, 2, score="softmax", groups=4, top_groups=1)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gaps_of_a_few_steps(score):
    """Pairs of experts whose values differ by -40 to 40 steps of 2^-24."""
    E, T = 128, 2000
    g = gen(7)
    base = torch.randn(1, E, generator=g) * 1.5
    x = base + torch.randint(-40, 41, (T, E), generator=g) * 2.0 ** -22
    s = scores(base, score)[0]
    bias = (0.5 - s).float()
    for k in (1, 4, 8, 10):
        agree(f"k {k}", x, bias, k, score=score)
        agree(f"k {k} in groups", x, bias, k, score=score, groups=8, top_groups=4)


@pytest.mark.parametrize("score", ["softmax"])
def test_a_softmax_total_that_rounds_down_at_every_step(score):
    """1024 experts, sixteen a lane: what 1 loses in its own lane's fifteen
    additions and in six steps across lanes, 20.7 steps of 2^-24 in all; the
    other expert's bias lies between the exact probability and 1."""
    u, E = 2.0 ** -24, 1024
    part = torch.empty(E, dtype=torch.float64)
    part[:16] = 0.99 * u
    for step in range(6):
        lanes = 2 ** step
        part[16 * lanes:32 * lanes] = 0.98 * u / (16 * lanes)
    x = torch.log(part).float()[None].repeat(4, 1)
    x[:, 0] = 0.0
    x[1:, 1:] += torch.tensor([-1e-3, -3e-3, -1e-2])[:, None]
    for n in range(12, 25):
        bias = torch.zeros(E)
        bias[E - 1] = 1.0 - n * u
        agree(f"total {n}", x, bias, 1, score=score)
        agree(f"total {n}, two", x, bias, 2, score=score)


# k up to 8 and above, 8 and 16 experts a lane, every number of lanes
@pytest.mark.parametrize("k", [1, 2, 4, 8, 9, 12])
@pytest.mark.parametrize("T,E", [(40, 16), (40, 64), (600, 64), (40, 100), (40, 256), (600, 256), (600, 130),
                                 (40, 512), (600, 512), (40, 1000)])
def test_zeros_of_both_signs_are_equal(T, E, k):
    """Logits of +0 and -0 across the last slot: equal ones by rising expert, with
    no bias, a bias of zeros and one of numbers, in both types, with and without
    groups."""
    g = gen(E + k)
    signs = torch.where(torch.rand(T, E, generator=g) < 0.5, 0.0, -0.0)
    x = torch.where(torch.rand(T, E, generator=g) < min(1.0, (k + 3) / E), signs, -1.0)
    x[0], x[1, :] = -0.0, -1.0
    x[1, 2], x[1, 5] = -0.0, 0.0
    x[2, :] = -1.0                        # k of +0, and one of -0 before them
    x[2, E - k:], x[2, 1] = 0.0, -0.0
    zeros = torch.where(torch.rand(E, generator=g) < 0.5, 0.0, -0.0)
    steps = torch.where(torch.rand(E, generator=g) < 0.5, 0.25, 0.5)
    for dtype in (F32, BF):
        for score in ("sigmoid", "softmax"):
            for bias in (None, zeros, steps):
                want, _ = choice(x, zeros if bias is None else bias, k, score)
                got = B.moe_route(x.to(dtype).to(DEV), k, score=score, scale=2.0, stats=False,
                                  bias=None if bias is None else bias.to(DEV)).idx.cpu().long()
                bad = (got != want).any(1).nonzero().flatten().tolist()
                assert not bad, (dtype, score, bias is None, bad[:3], got[bad[0]], want[bad[0]])
                if E % 4 == 0 and k <= E // 2:
                    want, _ = choice(x, zeros if bias is None else bias, k, score, 4, 2)
                    got = B.moe_route(x.to(dtype).to(DEV), k, score=score, groups=4, top_groups=2, stats=False,
                                      bias=None if bias is None else bias.to(DEV)).idx.cpu().long()
                    bad = (got != want).any(1).nonzero().flatten().tolist()
                    assert not bad, (dtype, score, "groups", bad[:3], got[bad[0]], want[bad[0]])


@pytest.mark.parametrize("k", [1, 3, 8, 10])
@pytest.mark.parametrize("T,E,groups", [(5, 64, 1), (5, 64, 4), (600, 128, 1), (600, 256, 8), (3, 512, 1)])
def test_nan_biases_beside_closed_ones(T, E, groups, k):
    """Biases of -inf for all but a few experts, and NaN of either sign: what is
    left is taken, a NaN never, also where nothing else is there to be compared."""
    x = torch.randn(T, E, generator=gen(E))
    for fine in (0, 1, 2):
        for score in ("sigmoid", "softmax"):
            bias = torch.full((E,), -INF)
            bias[7], bias[20] = math.nan, -math.nan
            bias[40:40 + fine] = 0.5
            r = B.moe_route(x.to(DEV), min(k, E // groups), score=score, groups=groups, bias=bias.to(DEV))
            idx = r.idx.cpu()
            assert not ((idx == 7) | (idx == 20)).any(), (fine, score)
            assert ((idx >= 0).sum(1) == min(fine, idx.shape[1])).all()
            assert (idx[idx >= 0] >= 40).all() and (idx[idx >= 0] < 40 + fine).all()
            assert int(r.counts[:E].sum()) == T * min(fine, idx.shape[1])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,groups,top_groups,best", [(65, 5, 5, 2, 2), (128, 6, 8, 3, 2), (160, 16, 8, 3, 1),
                                                        (256, 8, 8, 4, 2), (300, 10, 3, 2, 1), (512, 8, 16, 4, 2),
                                                        (512, 33, 8, 6, 2), (96, 8, 1, 1, 2)])
def test_from_1025_tokens_on_as_of_1024(E, k, groups, top_groups, best, score, dtype):
    """1024 tokens have eight experts a lane, 1025 sixteen: the same choices and
    counts, weights within the roundings of a total (21 steps of 2^-24) and of two
    scores and an inverse (5 steps), on both sides."""
    g = gen(E)
    x = (torch.randn(1025, E, generator=g) * 2).to(dtype)
    x[:, torch.randperm(E, generator=g)[:E // 9]] = -INF
    valid = torch.rand(1025, generator=g) < 0.9
    bias = torch.randn(E, generator=g) * 0.2
    for b in (bias, None, (bias * 8).round() / 8):
        kw = dict(score=score, bias=None if b is None else b.to(DEV), groups=groups, top_groups=top_groups,
                  group_best=best, scale=2.5)
        many = B.moe_route(x.to(DEV), k, valid=valid.to(DEV), **kw)
        few = B.moe_route(x[:1024].to(DEV), k, valid=valid[:1024].to(DEV), **kw)
        last = B.moe_route(x[1024:].to(DEV), k, valid=valid[1024:].to(DEV), **kw)
        assert torch.equal(many.idx, torch.cat([few.idx, last.idx]))
        assert torch.equal(many.counts, few.counts + last.counts)
        w = torch.cat([few.weights, last.weights])
        assert torch.all((many.weights - w).abs() <= 52 * 2.0 ** -24 * w)
        ps = few.prob_sum + last.prob_sum
        assert torch.all((many.prob_sum - ps).abs() <= (52 + 64) * 2.0 ** -24 * ps)
