"""GPU tests that the 8-bit products add in fp32, whatever the output's type and
however many rows there are.

Whole numbers whose products reach from 1 to 448^2 side by side (18 bits), with
the magnitudes of a sum below 2^24: every partial sum, in any order, is a whole
number that fp32 holds, so an fp32 result has to be the sum itself and a bf16
one the sum rounded once. An instruction that keeps fewer bits of a product
beside a larger one shows in many of them.

Random numbers: u = 2^-24, K products of a sum of magnitudes S add in fp32 with
at most 2 K u S (each addition may cut), fp32 block scales with two roundings
more; a bf16 result is off by another half step, 2^-8 of its value."""
import pytest
import torch

from decode_gemv_tensor_amd import binade as B

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
BF, F32, E4M3, E8M0 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def blocks(n):
    return -(-n // 128)


def mixed(shape, seed):
    """Whole numbers of four bits: most up to 15, some 256 to 448, of both signs."""
    g = gen(seed)
    small = torch.randint(-15, 16, shape, generator=g)
    large = torch.randint(8, 15, shape, generator=g) * 32 * (torch.randint(0, 2, shape, generator=g) * 2 - 1)
    return torch.where(torch.rand(shape, generator=g) < 0.05, large, small).float()


def exact_sum(a, b):
    """a b^T in fp64, after a look that fp32 holds every partial sum."""
    assert float((a.abs().double() @ b.abs().double().T).max()) < 2 ** 24
    return a.double() @ b.double().T


def weight(w, kind, train=False):
    """w in 8 bits with scales of one (a power of two or an fp32 number)."""
    s = torch.ones(*w.shape[:-2], blocks(w.shape[-2]), blocks(w.shape[-1]))
    return B.f8_weight(w.to(E4M3).to(DEV), (s if kind == "f32" else s.to(E8M0)).to(DEV), train=train)


def equal(name, got, want):
    bad = (got.cpu() != want.to(got.dtype)).sum().item()
    print(name, "differ:", bad, "of", want.numel(), flush=True)
    assert bad == 0, name


# 3000 x 4100 and 2048 x 6144: many tiles
@pytest.mark.parametrize("kind", ["e8m0", "f32"])
@pytest.mark.parametrize("m,n,k", [(3, 130, 416), (17, 40, 512), (40, 300, 416), (64, 257, 2080), (200, 300, 416),
                                   (260, 130, 1056), (3000, 4100, 384), (2048, 6144, 160)])
def test_gemm_adds_in_fp32(m, n, k, kind):
    x, w = mixed((m, k), 1), mixed((n, k), 2)
    want = exact_sum(x, w)
    for out in (BF, F32):
        equal(f"{out}", B.f8_gemm(x.to(BF).to(DEV), weight(w, kind), out_dtype=out), want)


@pytest.mark.parametrize("m,n,k", [(5, 300, 64), (16, 130, 160), (130, 416, 288), (416, 200, 96), (3000, 384, 4128)])
def test_gradients_add_in_fp32(m, n, k):
    x, dy, w = mixed((m, k), 3), mixed((m, n), 4), mixed((n, k), 5)
    if m > 416:                       # a sum over all rows has to stay below 2^24
        x[416:] = 0
    h = weight(w, "e8m0", True)
    want_dx, want_dw = exact_sum(dy, w.T), exact_sum(dy.T, x.T)
    for grads in (BF, F32):
        dx, dw = B.f8_gemm_grad(x.to(BF).to(DEV), h, dy.to(BF).to(DEV), grad_dtype=grads)
        equal("dx", dx, want_dx)
        equal(f"dw {grads}", dw, want_dw)


@pytest.mark.parametrize("kind", ["e8m0", "f32"])
@pytest.mark.parametrize("tokens,E,n", [(8, 4, 70), (200, 16, 130), (400, 9, 200), (900, 4, 257)])
def test_experts_add_in_fp32(tokens, E, n, kind):
    k, top = 416, 2
    x, w = mixed((tokens, k), 6), mixed((E, n, k), 7)
    idx = torch.randint(-1, E, (tokens, top), generator=gen(8)).int()
    want = torch.zeros(tokens * top, n, dtype=torch.float64)
    rows = x.repeat_interleave(top, 0)
    for e in range(E):
        at = idx.flatten() == e
        if at.any():
            want[at] = exact_sum(rows[at], w[e])
    for out in (BF, F32):
        equal(f"{out}", B.f8_moe_gemm(x.to(BF).to(DEV), weight(w, kind), idx.to(DEV), out_dtype=out), want)


@pytest.mark.parametrize("kind", ["e8m0", "f32"])
@pytest.mark.parametrize("m,n,k", [(40, 300, 1184), (200, 150, 4128), (2200, 4200, 544)])
def test_results_are_fp32_sums_rounded_once(m, n, k, kind):
    """Random values of e4m3, some much larger than the others."""
    g = gen(m)
    wide = lambda *shape: (torch.randn(*shape, generator=g) * torch.exp(2 * torch.randn(*shape, generator=g))).clamp(
        -448, 448)
    x, v = wide(m, k).to(E4M3).float(), wide(n, k).to(E4M3)
    x[:, ::128] = 448.0               # every block's scale is one: x is its own rounding
    s = torch.rand(blocks(n), blocks(k), generator=g) + 0.5
    s = s if kind == "f32" else (2.0 ** torch.floor(torch.log2(s))).to(E8M0)
    wd = v.double() * s.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    ref, absum = x.double() @ wd.T, x.double().abs() @ wd.abs().T
    h = B.f8_weight(v.to(DEV), s.to(DEV))
    for out in (BF, F32):
        y = B.f8_gemm(x.to(BF).to(DEV), h, out_dtype=out).cpu().double()
        tol = (2 * k + 4) * U * absum + (2.0 ** -8 * ref.abs() if out == BF else 0.0)
        worst = ((y - ref).abs() / tol).max().item()
        print(out, "worst", worst, flush=True)
        assert worst <= 1.0


def test_a_rows_result_is_the_same_sum_in_any_batch():
    """Sixteen rows alone and among others: both exact, so the same bits."""
    x, w = mixed((300, 416), 9), weight(mixed((260, 416), 10), "e8m0")
    few = B.f8_gemm(x[:16].to(BF).to(DEV), w, out_dtype=BF)
    for m in (17, 33, 65, 129, 300):
        assert torch.equal(B.f8_gemm(x[:m].to(BF).to(DEV), w, out_dtype=BF)[:16], few), m


@pytest.mark.parametrize("m", [3, 40])
def test_values_that_round_to_the_next_power_above_bf16(m):
    """255 2^120 in 8 bits is 2^128, which bf16 does not hold: infinite, in its row
    alone; 247 2^120 rounds down to 240 2^120."""
    x, w = mixed((m, 128), 11), mixed((40, 128), 12)
    w[:, 5] = w[:, 5].abs() + 1
    x[0, 5], x[1] = 255 * 2.0 ** 120, 0
    x[1, 5] = 247 * 2.0 ** 120
    w = w.clamp(-15, 15)
    clean = exact_sum(x.clamp(-448, 448), w)
    for out in (BF, F32):
        y = B.f8_gemm(x.to(BF).to(DEV), weight(w / 64, "e8m0"), out_dtype=out).cpu()
        assert bool((y[0] == torch.inf).all())
        assert torch.equal(y[1].double(), (240 * 2.0 ** 114 * w[:, 5].double()).to(out).double())
        assert torch.equal(y[2:], (clean[2:] / 64).to(out))
