"""GPU tests of the 8-bit products (binade_f8_pack, _layout, _gemm, _gemm_grad
and _moe_gemm) against their formulas.

Most inputs are small whole numbers times powers of two that change from block
to block: e4m3 holds them as they are, every sum of theirs is below 2^24 steps
and exact in fp32 (and a group of eight products spans fewer bits than the
8-bit matrix instruction keeps), so results have to be equal, a bf16 one to
the rounded sum. A wrong index, scale, block or mask shows.

Random inputs: u = 2^-24. Products of e4m3 values and powers of two are exact.
An fp32 output of K products then errs by at most K additions of two u each
(the matrix instruction may cut instead of rounding) of the sum S of the
products' magnitudes: 2 K u S; fp32 block scales add two roundings: 4 u S. The
8-bit instruction keeps 13 bits below the largest of eight products: each
loses less than 2^-12 of that one, at most 8 2^-12 in a group: below 2^-9 S on
the whole; a bf16 output adds half a step, 2^-9 of its value (within 2^-8)."""
import ctypes
import math

import pytest
import torch

from decode_gemv_tensor_amd import binade as B

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
BF, F32, E4M3, E8M0 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu


def say(*a):
    print(*a, flush=True)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def blocks(n):
    return -(-n // 128)


# ------------------------------------------------------------- the definition
def ref_q(v, whole_scale=None):
    """fp64 values of v quantised in blocks of 128 of the last axis, on the
    CPU, by rounding in 64 bits."""
    v = v.double()
    out = torch.zeros_like(v)
    for b in range(0, v.shape[-1], 128):
        p = v[..., b:b + 128]
        fin = torch.where(torch.isfinite(p), p, 0.0)
        top = fin.abs().amax(-1, keepdim=True)
        m, e = torch.frexp(top)
        e = torch.where(top > 0, e - 9 + (m > 0.875), 0).clamp(min=-126).double()
        out[..., b:b + 128] = ref_e4m3(p * 2.0 ** -e) * 2.0 ** e
    return out


def ref_e4m3(u):
    """fp64 u rounded to e4m3, ties to even; infinities and NaN become NaN."""
    fin = torch.where(torch.isfinite(u), u, 0.0)
    _, e = torch.frexp(fin.abs().clamp(min=2.0 ** -6))
    step = 2.0 ** (e.double() - 4)
    return torch.where(torch.isfinite(u), torch.round(fin / step) * step, math.nan)


def ref_w(values, scales):
    """fp64 of e4m3 values [..., N, K] and their blocks' scales."""
    n, k = values.shape[-2:]
    s = scales.float().double().repeat_interleave(128, -2)[..., :n, :]
    return values.float().double() * s.repeat_interleave(128, -1)[..., :k]


def whole_rows(m, k, seed, top=4):
    """bf16 [m, k] of whole numbers up to top, times a power of two for each
    block of a row; every block holds a +-top or nothing."""
    g = gen(seed)
    x = torch.randint(-top, top + 1, (m, k), generator=g).double()
    e = torch.randint(-2, 3, (m, blocks(k)), generator=g).double()
    return (x * (2.0 ** e).repeat_interleave(128, 1)[:, :k]).to(BF)


def whole_weight(count, n, k, seed, kind):
    """e4m3 values and scales whose products stay exact; some blocks zero."""
    g = gen(seed)
    v = torch.randint(-4, 5, (count, n, k), generator=g).float().to(E4M3)
    nb, kb = blocks(n), blocks(k)
    if kind == "f32":
        s = torch.randint(0, 6, (count, nb, kb), generator=g).float()
    else:
        s = (2.0 ** torch.randint(-2, 3, (count, nb, kb), generator=g)).float().to(E8M0)
    return (v[0], s[0]) if count == 1 else (v, s)


def equal(name, got, want):
    got = got.cpu()
    want = want.to(got.dtype)
    bad = got != want
    if bad.any():
        at = bad.nonzero()[0].tolist()
        say(name, "first difference at", at, float(got[tuple(at)]), "expected", float(want[tuple(at)]),
            int(bad.sum()), "of", bad.numel())
    assert not bad.any(), name


def near(name, got, ref, absum, k, exact, extra=4.0):
    """Within the bound above; NaN where (and only where) the formula has it: a
    random value that e4m3 does not reach is one."""
    got = got.cpu().double()
    assert torch.equal(got.isnan(), ref.isnan()), name
    got, ref, absum = got.nan_to_num(), ref.nan_to_num(), absum.nan_to_num()
    tol = (2 * k + extra) * U * absum
    if not exact:
        tol = tol + 2.0 ** -9 * absum
        tol = tol + 2.0 ** -8 * ref.abs()
    worst = ((got - ref).abs() / (tol + 1e-300)).max().item()
    say(name, "worst", worst)
    assert worst <= 1.0, name


SHAPES = [(1, 1, 32), (1, 17, 96), (3, 40, 128), (16, 130, 160), (17, 16, 32), (17, 130, 544),
          (31, 257, 1024), (33, 128, 1056), (64, 384, 2080), (65, 129, 288), (100, 1001, 640),
          (128, 128, 128), (129, 260, 1152), (300, 515, 416), (1, 1000, 4128), (5, 33, 15360)]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("kind", ["e8m0", "f32"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_whole_numbers(m, n, k, kind, out):
    say("gemm", m, n, k, kind, out)
    x = whole_rows(m, k, m + 7 * n)
    v, s = whole_weight(1, n, k, n + k, kind)
    y = B.f8_gemm(x.to(DEV), B.f8_weight(v.to(DEV), s.to(DEV)), out_dtype=out)
    equal("y", y, (x.double() @ ref_w(v, s).T).float())


@pytest.mark.parametrize("m,n,k", [(3000, 4100, 384), (2048, 6144, 1664)])
@pytest.mark.parametrize("kind", ["e8m0", "f32"])
def test_gemm_whole_numbers_large(m, n, k, kind):
    """Many tiles: the large tile, its edges and the order of the tiles."""
    say("gemm large", m, n, k, kind)
    x = whole_rows(m, k, 5)
    v, s = whole_weight(1, n, k, 6, kind)
    w = B.f8_weight(v.to(DEV), s.to(DEV))
    ref = (x.to(DEV).double() @ ref_w(v, s).to(DEV).T).float().cpu()
    for out in (BF, F32):
        equal(f"y {out}", B.f8_gemm(x.to(DEV), w, out_dtype=out), ref)


@pytest.mark.parametrize("m,n,k", [(2, 100, 416), (40, 300, 1184), (200, 150, 4128), (700, 3100, 640)])
@pytest.mark.parametrize("kind", ["e8m0", "f32"])
def test_gemm_random(m, n, k, kind):
    g = gen(m + k)
    x = (torch.randn(m, k, generator=g) * torch.exp(2 * torch.randn(m, 1, generator=g))).to(BF)
    v = (torch.randn(n, k, generator=g) * 100).to(E4M3)
    s = torch.rand(blocks(n), blocks(k), generator=g) + 0.1
    if kind == "e8m0":
        s = (2.0 ** torch.floor(torch.log2(s))).to(E8M0)
    q, w = ref_q(x), ref_w(v, s)
    ref, absum = q @ w.T, q.abs() @ w.abs().T
    h = B.f8_weight(v.to(DEV), s.to(DEV))
    near("fp32", B.f8_gemm(x.to(DEV), h), ref, absum, k, True)
    near("bf16", B.f8_gemm(x.to(DEV), h, out_dtype=BF), ref, absum, k, False)
    norm = (B.f8_gemm(x.to(DEV), h, out_dtype=BF).cpu().double() - ref).nan_to_num().norm() / \
        ref.nan_to_num().norm()
    assert norm <= 2.0 ** -9, norm          # half a bf16 step at most, and less on the whole


@pytest.mark.parametrize("grads", [BF, F32])
@pytest.mark.parametrize("m,n,k,kind", [(1, 1, 32, "e8m0"), (16, 40, 64, "f32"), (127, 129, 160, "e8m0"),
                                        (128, 200, 128, "f32"), (130, 64, 288, "e8m0"),
                                        (513, 1001, 416, "f32"), (1100, 136, 1056, "e8m0"),
                                        (260, 3000, 3200, "e8m0")])
def test_grad_whole_numbers(m, n, k, kind, grads):
    say("grad", m, n, k, kind, grads)
    x = whole_rows(k, m, 3).T.contiguous()       # powers of two along the rows t
    # dy: powers of two for blocks of columns (dx); of rows (dw)
    v, s = whole_weight(1, n, k, n + k, kind)
    w = B.f8_weight(v.to(DEV), s.to(DEV), train=True)
    dy = whole_rows(m, n, 4)
    dx, none = B.f8_gemm_grad(x.to(DEV), w, dy.to(DEV), need_dw=False)
    assert none is None
    equal("dx", dx, (dy.double() @ ref_w(v, s)).float())
    dy_t = whole_rows(n, m, 5).T.contiguous()
    none, dw = B.f8_gemm_grad(x.to(DEV), w, dy_t.to(DEV), need_dx=False, grad_dtype=grads)
    assert none is None
    equal("dw", dw, (dy_t.double().T @ x.double()).float())
    # both at once: plain whole numbers, whose blocks either way are exact
    g = gen(9)
    a = torch.randint(-4, 5, (m, k), generator=g).to(BF)
    b = torch.randint(-4, 5, (m, n), generator=g).to(BF)
    dx, dw = B.f8_gemm_grad(a.to(DEV), w, b.to(DEV), grad_dtype=grads)
    equal("dx of both", dx, (b.double() @ ref_w(v, s)).float())
    equal("dw of both", dw, (b.double().T @ a.double()).float())


@pytest.mark.parametrize("m,n,k", [(50, 70, 96), (300, 333, 544), (1000, 257, 800)])
def test_grad_random(m, n, k):
    g = gen(m)
    x = torch.randn(m, k, generator=g).to(BF)
    dy = (torch.randn(m, n, generator=g) * 1e-3 * torch.exp(torch.randn(m, 1, generator=g))).to(BF)
    v = (torch.randn(n, k, generator=g) * 100).to(E4M3)
    s = torch.rand(blocks(n), blocks(k), generator=g) * 1e-2
    w = B.f8_weight(v.to(DEV), s.to(DEV), train=True)
    dx, dw = B.f8_gemm_grad(x.to(DEV), w, dy.to(DEV))
    q, wd = ref_q(dy), ref_w(v, s)
    near("dx", dx, q @ wd, q.abs() @ wd.abs(), n, False)
    qt, xt = ref_q(dy.T.contiguous()), ref_q(x.T.contiguous())
    near("dw", dw, qt @ xt.T, qt.abs() @ xt.abs().T, m, True)


@pytest.mark.parametrize("count,n,k", [(1, 1, 32), (1, 128, 128), (1, 300, 416), (5, 130, 160), (3, 704, 256)])
def test_pack_is_the_definition(count, n, k):
    g = gen(n)
    w = (torch.randn(count, n, k, generator=g) * torch.exp(3 * torch.randn(count, n, 1, generator=g))).to(BF)
    w[0, 0, :8] = torch.tensor([0.0, -0.0, 2.0 ** -133, 1e30, -1e-30, 448.0, 3.0e-5, -1.0])
    if count == 1:
        w = w[0]
    p = B.f8_pack(w.to(DEV), train=True)
    K, N = blocks(k) * 128, blocks(n) * 128
    v = p.values.cpu().view(E4M3).view(count, K // 128, n, 128).transpose(1, 2).reshape(count, n, K).float().double()
    vt = p.values_t.cpu().view(E4M3).view(count, N // 128, k, 128).transpose(1, 2).reshape(count, k, N).float().double()
    nb, kb = blocks(n), blocks(k)
    s = p.scales.cpu().view(count, nb, -1)[:, :, :kb]
    st = p.scales_t.cpu().view(count, kb, -1)[:, :, :nb]
    assert torch.equal(st, s.transpose(1, 2))
    scale = 2.0 ** (s.double() - 127)
    for c in range(count):
        wc = w.view(count, n, k)[c].double()
        for i in range(nb):
            for j in range(kb):
                part = wc[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128]
                m, e = torch.frexp(part.abs().max())
                e = int(e) - 9 + int(m > 0.875) if m > 0 else 0
                e = max(e, -126)
                assert float(scale[c, i, j]) == 2.0 ** e
                want = ref_e4m3(part * 2.0 ** -e)
                r, l = part.shape
                assert torch.equal(v[c, i * 128:i * 128 + r, j * 128:j * 128 + l], want)
                assert torch.equal(vt[c, j * 128:j * 128 + l, i * 128:i * 128 + r], want.T)
    assert not v[:, :, k:].any() and not vt[:, :, n:].any()
    # again into the same planes, and of the packed weights through the product
    again = B.f8_pack(w.to(DEV), train=True, out=p)
    assert again is p


@pytest.mark.parametrize("x_per_slot", [False, True])
@pytest.mark.parametrize("tokens,E,top_k,n,k,kind,out", [
    (1, 4, 2, 40, 64, "e8m0", F32), (8, 128, 8, 70, 160, "e8m0", F32), (3, 5, 1, 257, 288, "f32", BF),
    (32, 2, 8, 33, 96, "f32", F32), (33, 8, 8, 130, 544, "e8m0", BF), (300, 16, 2, 200, 96, "f32", BF),
    (500, 7, 4, 129, 416, "e8m0", F32), (1000, 3, 1, 300, 160, "e8m0", BF), (700, 300, 4, 64, 32, "f32", F32)])
def test_experts_whole_numbers(tokens, E, top_k, n, k, kind, out, x_per_slot):
    say("experts", tokens, E, top_k, n, k, kind, out, x_per_slot)
    g = gen(tokens + E)
    rows = tokens * top_k if x_per_slot else tokens
    x = whole_rows(rows, k, 1)
    v, s = whole_weight(max(E, 2), n, k, 2, kind)
    v, s = v[:E], s[:E]
    idx = torch.randint(-1, E, (tokens, top_k), generator=g).to(torch.int32)
    idx[0, 0] = E - 1
    bad = idx.clone()
    bad[-1, -1] = E
    w = B.f8_weight(v.to(DEV), s.to(DEV))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = B.f8_moe_gemm(x.to(DEV), w, idx.to(DEV), x_per_slot=x_per_slot, out_dtype=out, status=status)
    assert int(status) == 0
    wd = ref_w(v, s)
    want = torch.zeros(tokens * top_k, n, dtype=torch.float64)
    flat = idx.flatten().long()
    xs = x.double() if x_per_slot else x.double().repeat_interleave(top_k, 0)
    for e in range(E):
        at = flat == e
        want[at] = xs[at] @ wd[e].T
    equal("y", y, want.float())
    y = B.f8_moe_gemm(x.to(DEV), w, bad.to(DEV), x_per_slot=x_per_slot, out_dtype=out, status=status)
    assert int(status) == B.DEV_BAD_INDEX
    want[-1] = 0
    equal("y with a bad index", y, want.float())
