"""GPU tests of the gradients of the experts' 8-bit products: expert by expert,
the rows of its pairs through f8_gemm_grad with weights of several experts.

Whole numbers that e4m3 holds, with sums below 2^24: results have to be equal to
the formulas'. Sizes whose experts' scales start at 4, 8 and 12 bytes past a
multiple of 16 are among them."""
import ctypes

import pytest
import torch

from decode_gemv_tensor_amd import binade as B

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32, E4M3, E8M0 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def whole(shape, seed, top=4):
    return torch.randint(-top, top + 1, shape, generator=gen(seed)).to(BF)


def blocks(n):
    return -(-n // 128)


def weights(E, n, k, seed, kind):
    """(handle with transposed planes, fp64 [E, n, k]), a scale of its own for each block."""
    g = gen(seed)
    v = torch.randint(-4, 5, (E, n, k), generator=g).float()
    s = torch.randint(1, 4, (E, blocks(n), blocks(k)), generator=g).float()
    s = s if kind == "f32" else 2.0 ** (s - 1)
    dense = v.double() * s.double().repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k]
    w = B.f8_weight(v.to(E4M3).to(DEV), (s if kind == "f32" else s.to(E8M0)).to(DEV), train=True)
    return w, dense


# codes of an expert: 5 x 12, 1 x 4, 2 x 4, 3 x 4 bytes, turned 10 x 8, 3 x 4, 2 x 4, 1 x 4
@pytest.mark.parametrize("kind", ["e8m0", "f32"])
@pytest.mark.parametrize("E,n,k", [(3, 640, 1280), (5, 70, 288), (4, 200, 160), (7, 300, 96), (1, 130, 64)])
def test_one_expert_of_several(E, n, k, kind):
    w, dense = weights(E, n, k, E + n, kind)
    for e in range(E):
        for m in (1, 9, 40):
            x, dy = whole((m, k), e + m), whole((m, n), e + m + 1, 2)
            for out in (F32, BF):
                y = B.f8_gemm(x.to(DEV), w, out_dtype=out, expert=e)
                assert torch.equal(y.cpu(), (x.double() @ dense[e].T).to(out)), (e, m, out)
            dx, dw = B.f8_gemm_grad(x.to(DEV), w, dy.to(DEV), expert=e)
            assert torch.equal(dx.cpu(), (dy.double() @ dense[e]).to(BF)), (e, m)
            assert torch.equal(dw.cpu(), (dy.double().T @ x.double()).float()), (e, m)
            none, dw = B.f8_gemm_grad(x.to(DEV), w, dy.to(DEV), need_dx=False, grad_dtype=BF, expert=e)
            assert none is None and torch.equal(dw.cpu(), (dy.double().T @ x.double()).to(BF))


@pytest.mark.parametrize("x_per_slot", [False, True])
@pytest.mark.parametrize("tokens,E,top_k,n,k", [(6, 4, 2, 70, 96), (150, 5, 3, 640, 160)])
def test_the_backward_of_the_experts_products(tokens, E, top_k, n, k, x_per_slot):
    """sum(y * dy) of f8_moe_gemm: dW of each expert, and dx summed over a token's
    slots, against the formulas and (whole numbers: exactly) against differences."""
    w, dense = weights(E, n, k, 3, "e8m0")
    rows = tokens * top_k if x_per_slot else tokens
    x, dy = whole((rows, k), 4, 2), whole((tokens * top_k, n), 5, 2)
    idx = torch.randint(-1, E - 1, (tokens, top_k), generator=gen(6)).int()   # the last expert has no pair
    xd, dyd, flat = x.to(DEV), dy.to(DEV), idx.flatten()
    dx = torch.zeros(tokens * top_k, k, dtype=BF, device=DEV)
    dw = torch.empty(E, n, k, device=DEV)
    for e in range(E):
        pairs = (flat == e).nonzero().flatten().to(DEV)
        xe = xd[pairs if x_per_slot else pairs // top_k]
        dx[pairs], _ = B.f8_gemm_grad(xe, w, dyd[pairs], expert=e, dw=dw[e])
    xs = x.double() if x_per_slot else x.double().repeat_interleave(top_k, 0)
    want_dx = torch.zeros(tokens * top_k, k, dtype=torch.float64)
    for e in range(E):
        at = flat == e
        want_dx[at] = dy[at].double() @ dense[e]
        assert torch.equal(dw[e].cpu(), (dy[at].double().T @ xs[at]).float())
    assert torch.equal(dx.cpu(), want_dx.to(BF))
    assert not bool(dw[E - 1].any())
    step = whole((rows, k), 7, 1)
    f = lambda a: float((B.f8_moe_gemm(a.to(DEV), w, idx.to(DEV), x_per_slot=x_per_slot).double() *
                         dyd.double()).sum())
    per_row = want_dx if x_per_slot else want_dx.view(tokens, top_k, k).sum(1)
    assert f(x + step) - f(x) == float((per_row * step.double()).sum())


def test_packed_again_and_replayed():
    """A graph of one expert's gradients reads the weights of its replay, not those
    of its capture."""
    E, n, k, m, e = 3, 640, 1280, 24, 1
    w0, w1 = whole((E, n, k), 1), whole((E, n, k), 2)
    x, dy = whole((m, k), 3).to(DEV), whole((m, n), 4, 2).to(DEV)
    w = B.f8_pack(w0.to(DEV), train=True)
    B.f8_gemm_grad(x, w, dy, expert=e)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dx, dw = B.f8_gemm_grad(x, w, dy, expert=e)
        y = B.f8_gemm(x, w, expert=e)
    for t in (w1 * 2, w0, w1, w0 * 4):
        B.f8_pack(t.to(DEV), train=True, out=w)
        graph.replay()
        torch.cuda.synchronize()
        d = t[e].double()
        assert torch.equal(y.cpu(), (x.cpu().double() @ d.T).float())
        assert torch.equal(dx.cpu(), (dy.cpu().double() @ d).to(BF))
        assert torch.equal(dw.cpu(), (dy.cpu().double().T @ x.cpu().double()).float())
        assert torch.equal(dx, B.f8_gemm_grad(x, w, dy, expert=e)[0])


def test_planes_of_one_expert_through_the_abi():
    """Where an expert's planes start: e / count of each plane's bytes on."""
    E, n, k, m = 4, 512, 512, 20            # 4 x 4 codes: a multiple of 16
    w, dense = weights(E, n, k, 8, "e8m0")
    x, dy = whole((m, k), 1).to(DEV), whole((m, n), 2, 2).to(DEV)
    st = torch.cuda.current_stream().cuda_stream
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())
    for e in range(E):
        at = [p.data_ptr() + p.numel() // E * e for p in (w.values, w.scales, w.values_t, w.scales_t)]
        d = B.F8Desc(n, k, 1, B.E8M0, *at)
        ws = torch.empty(B.lib().binade_f8_gemm_grad_workspace_bytes(m, n, k, 1, 0, B.F32), dtype=torch.uint8,
                         device=DEV)
        dx = torch.empty(m, k, dtype=BF, device=DEV)
        assert B.lib().binade_f8_gemm_grad(ctypes.byref(d), None, m, k, ptr(dy), n, ptr(dx), k, None, B.F32,
                                           ptr(ws), ws.numel(), st) == B.OK
        assert torch.equal(dx.cpu(), (dy.cpu().double() @ dense[e]).to(BF))
    assert torch.equal(B.f8_gemm(x, w, expert=2).cpu(), (x.cpu().double() @ dense[2].T).float())


def test_refusals():
    w, _ = weights(3, 70, 96, 1, "e8m0")
    x, dy = whole((4, 96), 1).to(DEV), whole((4, 70), 2).to(DEV)
    for e in (-1, 3):
        with pytest.raises(ValueError, match="expert"):
            B.f8_gemm(x, w, expert=e)
        with pytest.raises(ValueError, match="expert"):
            B.f8_gemm_grad(x, w, dy, expert=e)
    with pytest.raises(TypeError):
        B.f8_gemm(x, w, expert=1.0)
    with pytest.raises(B.BinadeError):       # several experts, and none said
        B.f8_gemm(x, w)
    with pytest.raises(B.BinadeError):
        B.f8_gemm_grad(x, w, dy)
    v = torch.zeros(3, 70, 96).to(E4M3).to(DEV)
    plain = B.f8_weight(v, torch.ones(3, 1, 1, device=DEV))
    with pytest.raises(B.BinadeError):       # no transposed planes
        B.f8_gemm_grad(x, plain, dy, expert=0)
    dx, dw = B.f8_gemm_grad(x, plain, dy, expert=0, need_dx=False)
    assert dx is None and dw.shape == (70, 96)
