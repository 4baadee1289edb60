"""GPU tests of the 8-bit products and the router by scores as they are used:
together, on several streams, in graphs, with exact workspaces, strided rows
and special values.

Whole numbers as in the products' own tests: results have to be equal. A layer
is checked stage by stage, each against 64 bits from the stage before: K
products of e4m3 values and powers of two err by at most 2 K u S (u = 2^-24, S
the sum of their magnitudes); a bf16 result through the 8-bit instruction by
2^-9 S and half a step, 2^-9 of its value, more (within 2^-8)."""
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


def q8(v):
    """fp64 values of v in 8 bits with a power of two for each 128 of a row."""
    v = v.double()
    out = torch.zeros_like(v)
    for b in range(0, v.shape[-1], 128):
        p = v[..., b:b + 128]
        top = torch.where(torch.isfinite(p), p, 0.0).abs().amax(-1, keepdim=True)
        m, e = torch.frexp(top)
        e = torch.where(top > 0, e - 9 + (m > 0.875), 0).clamp(min=-126).double()
        u = p * 2.0 ** -e
        fin = torch.where(torch.isfinite(u), u, 0.0)
        step = 2.0 ** (torch.frexp(fin.abs().clamp(min=2.0 ** -6))[1].double() - 4)
        out[..., b:b + 128] = torch.where(torch.isfinite(u), torch.round(fin / step) * step * 2.0 ** e, math.nan)
    return out


def whole(m, k, seed, top=4):
    return torch.randint(-top, top + 1, (m, k), generator=gen(seed)).to(BF)


def whole_w(count, n, k, seed, kind="e8m0"):
    g = gen(seed)
    v = torch.randint(-4, 5, (count, n, k), generator=g).float().to(E4M3)
    s = torch.randint(0, 3, (count, blocks(n), blocks(k)), generator=g).float()
    s = s if kind == "f32" else (2.0 ** (s - 1)).to(E8M0)
    return (v[0], s[0]) if count == 1 else (v, s)


def dense(v, s):
    n, k = v.shape[-2:]
    s = s.float().double().repeat_interleave(128, -2)[..., :n, :]
    return v.float().double() * s.repeat_interleave(128, -1)[..., :k]


# ------------------------------------------------------------- through the ABI
def abi_gemm(w, x, ldx, m, y, ldy, dt, ws, nb):
    st = torch.cuda.current_stream().cuda_stream
    return B.lib().binade_f8_gemm(ctypes.byref(w.desc()), P(x), m, ldx, P(y), ldy, dt, P(ws), nb, st)


def P(t):
    return None if t is None else ctypes.c_void_p(t if isinstance(t, int) else t.data_ptr())


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("m,n,k", [(1, 130, 288), (16, 33, 96), (17, 33, 96), (70, 300, 1056), (200, 129, 2080),
                                   (2100, 5000, 160)])
def test_gemm_strides_exact_workspace_and_what_lies_behind(m, n, k, out):
    """Rows at odd strides and offsets, the workspace to its last byte: bytes
    behind it, columns behind N and rows behind m stay as they were."""
    say("strides", m, n, k, out)
    x = whole(m, k, 1)
    v, s = whole_w(1, n, k, 2)
    w = B.f8_weight(v.to(DEV), s.to(DEV))
    wide = torch.full((m, k + 24), 7.0, dtype=BF, device=DEV)
    wide[:, 8:8 + k] = x.to(DEV)
    code = 1 if out == BF else 0
    need = B.lib().binade_f8_gemm_workspace_bytes(m, n, k, code)
    ws = torch.full((need + 512,), 0xAB, dtype=torch.uint8, device=DEV)
    want = (x.to(DEV).double() @ dense(v, s).to(DEV).T).to(out)
    for off, ldy in ((0, n), (1, n + 3), (8, (n + 15) // 8 * 8)):
        flat = torch.full((off + (m + 2) * ldy,), 9.0, dtype=out, device=DEV)
        y = flat[off:].view(m + 2, ldy)
        assert abi_gemm(w, wide[:, 8:], k + 24, m, y, ldy, code, ws, need) == B.OK
        torch.cuda.synchronize()
        assert torch.equal(y[:m, :n], want)
        assert bool((y[m:] == 9).all()) and bool((y[:, n:] == 9).all()) and bool((flat[:off] == 9).all())
        assert bool((ws[need:] == 0xAB).all())


@pytest.mark.parametrize("grads", [BF, F32])
@pytest.mark.parametrize("m,n,k", [(1, 7, 32), (130, 257, 96), (257, 100, 416)])
def test_grad_strides_and_exact_workspace(m, n, k, grads):
    say("grad strides", m, n, k, grads)
    x, dy = whole(m, k, 1), whole(m, n, 2)
    v, s = whole_w(1, n, k, 3)
    w = B.f8_weight(v.to(DEV), s.to(DEV), train=True)
    xw = torch.full((m, k + 8), 5.0, dtype=BF, device=DEV)
    xw[:, :k] = x.to(DEV)
    dyw = torch.full((m * (n + 5) + 1,), 5.0, dtype=BF, device=DEV)
    dyv = dyw[1:].view(m, n + 5)                     # rows at every alignment
    dyv[:, :n] = dy.to(DEV)
    code = 1 if grads == BF else 0
    need = B.lib().binade_f8_gemm_grad_workspace_bytes(m, n, k, 1, 1, code)
    ws = torch.full((need + 512,), 0xAB, dtype=torch.uint8, device=DEV)
    dx = torch.full((m + 1, k + 3), 9.0, dtype=BF, device=DEV)
    dw = torch.full((n + 1, k), 9.0, dtype=grads, device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    assert B.lib().binade_f8_gemm_grad(ctypes.byref(w.desc()), P(xw), m, k + 8, P(dyv), n + 5, P(dx), k + 3, P(dw),
                                       code, P(ws), need, st) == B.OK
    torch.cuda.synchronize()
    assert torch.equal(dx[:m, :k].cpu(), (dy.double() @ dense(v, s)).to(BF))
    assert torch.equal(dw[:n].cpu(), (dy.double().T @ x.double()).to(grads))
    assert bool((dx[m:] == 9).all()) and bool((dx[:, k:] == 9).all()) and bool((dw[n:] == 9).all())
    assert bool((ws[need:] == 0xAB).all())


@pytest.mark.parametrize("tokens,top_k", [(8, 2), (100, 6), (1500, 3)])
def test_experts_exact_workspace(tokens, top_k):
    E, n, k = 20, 70, 160
    x = whole(tokens, k, 1)
    v, s = whole_w(E, n, k, 2)
    idx = torch.randint(-1, E, (tokens, top_k), generator=gen(3)).int()
    w = B.f8_weight(v.to(DEV), s.to(DEV))
    need = B.lib().binade_f8_moe_workspace_bytes(tokens, top_k, 0, E, n, k)
    ws = torch.full((need + 512,), 0xAB, dtype=torch.uint8, device=DEV)
    xd, idd = x.to(DEV), idx.to(DEV)
    pairs = tokens * top_k
    y = torch.full((pairs + 2, n + 5), 9.0, device=DEV)
    st = torch.cuda.current_stream().cuda_stream
    assert B.lib().binade_f8_moe_gemm(ctypes.byref(w.desc()), P(xd), k, 0, P(idd), tokens, top_k, P(y), n + 5, 0,
                                      P(ws), need, None, st) == B.OK
    torch.cuda.synchronize()
    wd = dense(v, s)
    want = torch.zeros(pairs, n, dtype=torch.float64)
    rows = x.double().repeat_interleave(top_k, 0)
    for e in range(E):
        at = idx.flatten() == e
        want[at] = rows[at] @ wd[e].T
    assert torch.equal(y[:pairs, :n].cpu(), want.float())
    assert bool((y[pairs:] == 9).all()) and bool((y[:, n:] == 9).all()) and bool((ws[need:] == 0xAB).all())


@pytest.mark.parametrize("idx_of", ["one", "none", "last", "each"])
@pytest.mark.parametrize("tokens", [30, 400])
def test_experts_uneven_choices(tokens, idx_of):
    """All pairs with one expert, none with any, the last expert's, one each."""
    E, n, k, top_k = 13, 200, 96, 4
    idx = {"one": torch.zeros(tokens, top_k), "none": torch.full((tokens, top_k), -1),
           "last": torch.full((tokens, top_k), E - 1),
           "each": torch.arange(tokens * top_k).view(tokens, top_k) % E}[idx_of].int()
    x = whole(tokens, k, 5)
    v, s = whole_w(E, n, k, 6, "f32")
    wd = dense(v, s)
    w = B.f8_weight(v.to(DEV), s.to(DEV))
    for out in (BF, F32):
        y = B.f8_moe_gemm(x.to(DEV), w, idx.to(DEV), out_dtype=out)
        rows = x.double().repeat_interleave(top_k, 0)
        want = torch.zeros(tokens * top_k, n, dtype=torch.float64)
        for e in range(E):
            at = idx.flatten() == e
            want[at] = rows[at] @ wd[e].T
        assert torch.equal(y.cpu(), want.to(out))


def test_nothing_to_do():
    v, s = whole_w(1, 40, 64, 1)
    w = B.f8_weight(v.to(DEV), s.to(DEV), train=True)
    none = torch.empty(0, 64, dtype=BF, device=DEV)
    assert B.f8_gemm(none, w).shape == (0, 40)
    dx, dw = B.f8_gemm_grad(none, w, torch.empty(0, 40, dtype=BF, device=DEV))
    assert dx.shape == (0, 64) and dw.shape == (40, 64) and not bool(dw.any())
    dx, dw = B.f8_gemm_grad(none, w, torch.empty(0, 40, dtype=BF, device=DEV), grad_dtype=BF, need_dx=False)
    assert dx is None and not bool(dw.any())
    v, s = whole_w(3, 40, 64, 1)
    e = B.f8_weight(v.to(DEV), s.to(DEV))
    assert B.f8_moe_gemm(none, e, torch.empty(0, 2, dtype=torch.int32, device=DEV)).shape == (0, 40)


# ------------------------------------------------------------- special values
@pytest.mark.parametrize("m,n,k,out", [(1, 300, 416, F32), (9, 300, 416, BF), (20, 300, 416, F32),
                                       (20, 300, 416, BF), (300, 200, 1056, BF), (300, 200, 1056, F32),
                                       (2100, 5000, 160, BF)])
def test_infinities_and_nan_stay_in_their_rows_and_columns(m, n, k, out):
    x = whole(m, k, 1)
    v, s = whole_w(1, n, k, 2)
    clean = (x.to(DEV).double() @ dense(v, s).to(DEV).T).to(out).cpu()
    bad = x.clone()
    bad[m - 1, 5] = math.inf
    if m > 2:
        bad[0, k - 1] = math.nan
        bad[m // 2, 0] = -math.inf
    rows = sorted({m - 1} | ({0, m // 2} if m > 2 else set()))
    y = B.f8_gemm(bad.to(DEV), B.f8_weight(v.to(DEV), s.to(DEV)), out_dtype=out).cpu()
    keep = torch.ones(m, dtype=torch.bool)
    keep[rows] = False
    assert bool(y[rows].isnan().all()) and torch.equal(y[keep], clean[keep])
    # a NaN among the weights: its column; among the scales: its block's columns
    vb = v.view(torch.uint8).clone()
    vb[n - 1, k - 1] = 0x7F
    vb[3, 0] = 0xFF
    y = B.f8_gemm(x.to(DEV), B.f8_weight(vb.view(E4M3).to(DEV), s.to(DEV)), out_dtype=out).cpu()
    keep = torch.ones(n, dtype=torch.bool)
    keep[[3, n - 1]] = False
    assert bool(y[:, ~keep].isnan().all()) and torch.equal(y[:, keep], clean[:, keep])
    for bits in (s.view(torch.uint8), s.float()):
        sb = bits.clone()
        sb[1, 0] = 255 if bits.dtype == torch.uint8 else math.nan
        y = B.f8_gemm(x.to(DEV), B.f8_weight(v.to(DEV), sb.to(DEV)), out_dtype=out).cpu()
        keep = torch.ones(n, dtype=torch.bool)
        keep[128:256] = False
        assert bool(y[:, ~keep].isnan().all()) and torch.equal(y[:, keep], clean[:, keep])


@pytest.mark.parametrize("m,out", [(2, F32), (2, BF), (40, F32), (40, BF)])
def test_smallest_and_large_scales(m, out):
    """Codes 0 (2^-127) and 240, the fp32 scales 2^-140 and 2^100, beside rows of
    x that bring the products back into range."""
    n, k = 130, 256
    x = whole(m, k, 1)
    v = torch.randint(-4, 5, (n, k), generator=gen(2)).float().to(E4M3)
    for up, sc in ((100, torch.full((2, 2), 0, dtype=torch.uint8)), (-100, torch.full((2, 2), 240, dtype=torch.uint8)),
                   (100, torch.full((2, 2), 2.0 ** -140)), (-100, torch.full((2, 2), 2.0 ** 100))):
        real = 2.0 ** (sc.double() - 127) if sc.dtype == torch.uint8 else sc.double()
        xs = (x.double() * 2.0 ** up).to(BF)
        y = B.f8_gemm(xs.to(DEV), B.f8_weight(v.to(DEV), sc.to(DEV)), out_dtype=out)
        want = (xs.double() @ v.float().double().T) * real[0, 0]
        assert torch.equal(y.cpu(), want.to(out)), (up, sc.dtype)


def test_grad_of_infinities_and_nan():
    m, n, k = 150, 140, 96
    x, dy = whole(m, k, 1), whole(m, n, 2)
    v, s = whole_w(1, n, k, 3)
    w = B.f8_weight(v.to(DEV), s.to(DEV), train=True)
    dx0, dw0 = (t.cpu() for t in B.f8_gemm_grad(x.to(DEV), w, dy.to(DEV)))
    dy[7, 130] = math.inf
    x[140, 3] = math.nan
    dx, dw = (t.cpu() for t in B.f8_gemm_grad(x.to(DEV), w, dy.to(DEV)))
    assert bool(dx[7].isnan().all())
    dx[7] = dx0[7]
    assert torch.equal(dx, dx0)
    assert bool(dw[130].isnan().all()) and bool(dw[:, 3].isnan().all())
    dw[130], dw[:, 3] = dw0[130], dw0[:, 3]
    assert torch.equal(dw, dw0)


def test_grad_against_differences():
    """Whole numbers: f(x + e) - f(x) is sum(dx * e), all exact."""
    m, n, k = 40, 70, 160
    v, s = whole_w(1, n, k, 4)
    w = B.f8_weight(v.to(DEV), s.to(DEV), train=True)
    x, dy = whole(m, k, 5).to(DEV), whole(m, n, 6).to(DEV)
    dx, dw = B.f8_gemm_grad(x, w, dy)
    f = lambda a, b: float((B.f8_gemm(a, b).double() * dy.double()).sum())
    e = whole(m, k, 7, 1).to(DEV)
    # dx is a bf16: its sums are whole numbers up to 70 * 4 * 4 * 2, which it may round
    exact = dy.double() @ dense(v, s).to(DEV)
    assert f(x + e, w) - f(x, w) == float((exact * e.double()).sum())
    assert torch.equal(dx, exact.to(BF))
    ev = torch.randint(-1, 2, (n, k), generator=gen(8)).float().clamp(-4, 4)
    v2 = (v.float() + ev).to(E4M3)
    step = f(x, B.f8_weight(v2.to(DEV), s.to(DEV))) - f(x, w)
    assert step == float((dw.double() * (dense(v2, s) - dense(v, s)).to(DEV)).sum())


# ------------------------------------------------------------- streams, graphs
def small_layer(d, stream=None):
    r = B.moe_route(d["logits"], 4, score="sigmoid", bias=d["bias"], groups=4, top_groups=2, scale=2.5, stream=stream)
    g = B.f8_moe_gemm(d["x"], d["gate"], r.idx, stream=stream)
    u = B.f8_moe_gemm(d["x"], d["up"], r.idx, stream=stream)
    h = B.moe_silu_mul(g, u, stream=stream)
    y = B.f8_moe_gemm(h, d["down"], r.idx, x_per_slot=True, stream=stream)
    o = B.moe_combine(y, r.weights, 4, out_dtype=BF, stream=stream)
    _, dw = B.moe_combine_grad(y, r.weights, d["dout"], 4, stream=stream)
    dl = B.moe_route_grad(d["logits"], r.idx, dweights=dw, counts=r.counts, dloss=d["one"], score="sigmoid",
                          scale=2.5, stream=stream)
    p = B.f8_gemm(d["x"], d["dense"], out_dtype=BF, stream=stream)
    dx, dwt = B.f8_gemm_grad(d["x"], d["dense"], d["dy"], stream=stream)
    return r.idx, r.weights, r.counts, r.loss, g, u, h, y, o, dl, p, dx, dwt


def layer_data(T, seed, E=16, hid=160, ffn=96, n=200):
    g = gen(seed)
    pack = lambda *shape: B.f8_pack((torch.randn(*shape, generator=g) * 0.1).to(BF).to(DEV), train=True)
    return {"logits": torch.randn(T, E, generator=g).to(DEV), "bias": (torch.randn(E, generator=g) * 0.1).to(DEV),
            "x": torch.randn(T, hid, generator=g).to(BF).to(DEV), "gate": pack(E, ffn, hid), "up": pack(E, ffn, hid),
            "down": pack(E, hid, ffn), "dense": pack(n, hid), "dy": torch.randn(T, n, generator=g).to(BF).to(DEV),
            "dout": torch.randn(T, hid, generator=g).to(DEV), "one": torch.ones(1, device=DEV)}


@pytest.mark.parametrize("T", [3, 90, 400])
def test_streams_and_graphs(T):
    """Two streams at once and a graph replayed with other data, eager work in
    between: the same bits as one call after the other."""
    data = [layer_data(T, 10 + s) for s in range(3)]
    want = [small_layer(d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = [small_layer(d, s) for d, s in zip(data, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(i, j) for i, j in zip(a, b))
    buf = {key: t.clone() if isinstance(t, torch.Tensor) else
           B.F8Weight(t.rows, t.cols, t.count, t.scale_dtype, t.values.clone(), t.scales.clone(), t.values_t.clone(),
                      t.scales_t.clone()) for key, t in data[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = small_layer(buf)
    for j in (1, 2, 0, 1, 2):
        for key, t in data[j].items():
            if isinstance(t, torch.Tensor):
                buf[key].copy_(t)
            else:
                for plane in ("values", "scales", "values_t", "scales_t"):
                    getattr(buf[key], plane).copy_(getattr(t, plane))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[j])), j
        small_layer(data[j])


def test_two_graphs_with_workspaces_of_their_own():
    """Two graphs replayed on two streams at once, each with its workspace; then
    one workspace for calls one after the other."""
    m, n, k = 300, 260, 544
    v, s = whole_w(1, n, k, 1)
    w = B.f8_weight(v.to(DEV), s.to(DEV))
    xs = [whole(m, k, 2 + i).to(DEV) for i in range(2)]
    want = [(x.double() @ dense(v, s).to(DEV).T).float() for x in xs]
    need = B.lib().binade_f8_gemm_workspace_bytes(m, n, k, B.F32)
    ws = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in range(2)]
    graphs, ys = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ys.append(B.f8_gemm(xs[i], w, workspace=ws[i]))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        torch.cuda.synchronize()
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        for st, graph in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, t) for y, t in zip(ys, want))
    for _ in range(3):
        for i in range(2):
            assert torch.equal(B.f8_gemm(xs[i], w, workspace=ws[0]), want[i])


# ------------------------------------------------------------- together
def close(name, got, ref, absum, k, eight_bits):
    got = got.detach().cpu().double()
    tol = (2 * k + 4) * U * absum
    if eight_bits:
        tol = tol + 2.0 ** -9 * absum + 2.0 ** -8 * ref.abs()
    worst = ((got - ref).abs() / (tol + 1e-30)).max().item()
    say(name, "worst", worst)
    assert worst <= 1.0, name


@pytest.mark.parametrize("T", [5, 120])
def test_a_layer_of_experts_by_scores(T):
    """Router by scores -> gate and up -> SiLU * up -> down -> combine, each
    stage from the one before, and back to the logits."""
    E, top, hid, ffn = 16, 4, 160, 288
    g = gen(3)
    ws = [(torch.randn(E, *shape, generator=g) * 0.1).to(BF) for shape in ((ffn, hid), (ffn, hid), (hid, ffn))]
    gate, up, down = (B.f8_pack(w.to(DEV)) for w in ws)
    real = []
    for w, p in zip(ws, (gate, up, down)):     # the planes are the weights' own, block by block
        rows, cols = w.shape[1:]
        val = p.values.view(E4M3).view(E, blocks(cols), rows, 128).transpose(1, 2).reshape(E, rows, -1)
        sc = 2.0 ** (p.scales.view(E, blocks(rows), -1)[:, :, :blocks(cols)].cpu().double() - 127)
        val = val[:, :, :cols].float().cpu().double() * sc.repeat_interleave(128, 1)[:, :rows].repeat_interleave(
            128, 2)[:, :, :cols]
        assert torch.all((val - w.double()).abs() <= 2.0 ** -4 * w.double().abs() + 2.0 ** -10 * sc.max())
        real.append(val)
    x = torch.randn(T, hid, generator=g).to(BF)
    logits = torch.randn(T, E, generator=g)
    bias = torch.randn(E, generator=g) * 0.1
    r = B.moe_route(logits.to(DEV), top, score="sigmoid", bias=bias.to(DEV), groups=4, top_groups=2, scale=2.5)
    sig = torch.sigmoid(logits.double())
    val = sig + bias.double()
    grp = val.view(T, 4, 4).topk(2, -1).values.sum(-1)
    keep = torch.zeros(T, 4, dtype=torch.bool).scatter_(1, grp.topk(2, -1).indices, True).repeat_interleave(4, 1)
    idx = val.masked_fill(~keep, -math.inf).topk(top, -1).indices
    assert torch.equal(r.idx.cpu().long(), idx)
    taken = sig.gather(1, idx)
    weights = 2.5 * taken / taken.sum(1, keepdim=True)
    D = 2 * float(logits.abs().max())
    assert torch.all((r.weights.cpu().double() - weights).abs() <= (4 * D + 64) * U * weights)
    flat = idx.flatten()

    def experts(rows, w):
        prod = lambda a, b: torch.stack([b[e] @ a[p] for p, e in enumerate(flat.tolist())])
        q = q8(rows)
        return prod(q, w), prod(q.abs(), w.abs())

    slots = x.repeat_interleave(top, 0)
    ga, ua = (B.f8_moe_gemm(x.to(DEV), p, r.idx) for p in (gate, up))
    close("gate", ga, *experts(slots, real[0]), hid, False)
    close("up", ua, *experts(slots, real[1]), hid, False)
    h = B.moe_silu_mul(ga, ua)
    y = B.f8_moe_gemm(h, down, r.idx, x_per_slot=True)
    close("down", y, *experts(h.cpu(), real[2]), ffn, False)
    yb = B.f8_moe_gemm(h, down, r.idx, x_per_slot=True, out_dtype=BF)
    close("down in bf16", yb, *experts(h.cpu(), real[2]), ffn, True)
    o = B.moe_combine(y, r.weights, top)
    part = (y.cpu().double() * r.weights.cpu().double().view(-1, 1)).view(T, top, hid)
    close("combine", o, part.sum(1), part.abs().sum(1), top, False)
    # back to the logits: the weights' gradient through the choice that was made
    dout = torch.randn(T, hid, generator=g)
    _, dw = B.moe_combine_grad(y, r.weights, dout.to(DEV), top)
    dl = B.moe_route_grad(logits.to(DEV), r.idx, dweights=dw, score="sigmoid", bias=bias.to(DEV), groups=4, scale=2.5)
    z = logits.double().requires_grad_()
    t = torch.sigmoid(z).gather(1, idx)
    (2.5 * t / t.sum(1, keepdim=True) * dw.cpu().double()).sum().backward()
    big = (2.5 * dw.cpu().double().abs().sum(1, keepdim=True)).expand_as(z)
    assert torch.all((dl.cpu().double() - z.grad).abs() <= (8 * D + 128) * U * big)


def test_a_training_step_of_a_projection():
    """f8_pack -> f8_gemm -> f8_gemm_grad -> an update -> f8_pack into the same
    planes -> f8_gemm."""
    m, n, k = 200, 264, 416
    g = gen(5)
    w = (torch.randn(n, k, generator=g) * 0.05).to(BF)
    x, dy = (torch.randn(m, c, generator=g).to(BF) for c in (k, n))
    p = B.f8_pack(w.to(DEV), train=True)
    tile = lambda t: torch.cat([torch.cat([qb(c) for c in r.split(128, 1)], 1) for r in t.double().split(128, 0)], 0)

    def qb(block):                                   # a 128 x 128 block as one row of any length
        top = block.abs().max()
        mant, e = torch.frexp(top)
        e = max(int(e) - 9 + int(mant > 0.875), -126) if top > 0 else 0
        u = block * 2.0 ** -e
        step = 2.0 ** (torch.frexp(u.abs().clamp(min=2.0 ** -6))[1].double() - 4)
        return torch.round(u / step) * step * 2.0 ** e

    for _ in range(2):
        wd, q = tile(w), q8(x)
        close("y fp32", B.f8_gemm(x.to(DEV), p), q @ wd.T, q.abs() @ wd.abs().T, k, False)
        close("y bf16", B.f8_gemm(x.to(DEV), p, out_dtype=BF), q @ wd.T, q.abs() @ wd.abs().T, k, True)
        dx, dw = B.f8_gemm_grad(x.to(DEV), p, dy.to(DEV))
        qd = q8(dy)
        close("dx", dx, qd @ wd, qd.abs() @ wd.abs(), n, True)
        a, b = q8(dy.T.contiguous()), q8(x.T.contiguous())
        close("dw", dw, a @ b.T, a.abs() @ b.abs().T, m, False)
        w = (w.float() - 1e-3 * dw.cpu()).to(BF)
        assert B.f8_pack(w.to(DEV), train=True, out=p) is p


def test_bindings_refuse():
    v, s = whole_w(1, 40, 64, 1)
    w = B.f8_weight(v.to(DEV), s.to(DEV))
    x = whole(4, 64, 1).to(DEV)
    with pytest.raises(TypeError):
        B.f8_gemm(x.float(), w)
    with pytest.raises(ValueError):
        B.f8_gemm(x[:, :32], w)
    with pytest.raises(TypeError):
        B.f8_gemm(x, v.to(DEV))
    with pytest.raises(ValueError):
        B.f8_gemm(whole(40, 64, 1).to(DEV), w, workspace=torch.empty(64, 64, dtype=torch.uint8, device=DEV).T)
    with pytest.raises(B.BinadeError):
        B.f8_gemm(whole(40, 64, 1).to(DEV), w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(B.BinadeError):
        B.f8_gemm_grad(x, w, whole(4, 40, 2).to(DEV))          # no transposed planes
    with pytest.raises(ValueError):
        B.f8_gemm_grad(x, w, whole(4, 41, 2).to(DEV), need_dx=False)
    with pytest.raises(TypeError):
        B.f8_weight(v.float().to(DEV), s.to(DEV))
    with pytest.raises(ValueError):
        B.f8_weight(v.to(DEV), s[:0].to(DEV))
    with pytest.raises(ValueError):
        B.f8_moe_gemm(x, w, torch.zeros(4, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        B.f8_moe_gemm(x, w, torch.zeros(5, 1, dtype=torch.int32, device=DEV))
    # x rows that the call does not take as they lie are copied
    odd = torch.zeros(4, 70, dtype=BF, device=DEV)
    odd[:, 3:67] = x
    assert torch.equal(B.f8_gemm(odd[:, 3:67], w), B.f8_gemm(x, w))


# ------------------------------------------------------------- far offsets
@pytest.mark.parametrize("m,n,k,out", [(1 << 20, 16, 4224, BF), (1 << 20, 16, 4224, F32), (1 << 20, 4200, 32, F32)])
def test_rows_past_32_bits_of_bytes(m, n, k, out):
    """Rows that repeat: every period's results are those of the first rows alone."""
    say("far rows", m, n, k, out)
    base = whole(4096, k, 1)
    v, s = whole_w(1, n, k, 2)
    w = B.f8_weight(v.to(DEV), s.to(DEV))
    want = (base.double() @ dense(v, s).T).to(out).to(DEV)
    x = base.to(DEV).repeat(m // 4096, 1)
    assert x.numel() * 2 > 1 << 32 or m * n * 4 > 1 << 32
    y = B.f8_gemm(x, w, out_dtype=out).view(-1, 4096, n)
    assert all(torch.equal(y[i], want) for i in range(y.shape[0]))


def test_gradients_past_32_bits_of_bytes():
    m, n, k = 1 << 20, 32, 4224
    base, dyb = whole(4096, k, 1, 1), whole(4096, n, 2, 1)
    v, s = whole_w(1, n, k, 3)
    w = B.f8_weight(v.to(DEV), s.to(DEV), train=True)
    x, dy = base.to(DEV).repeat(m // 4096, 1), dyb.to(DEV).repeat(m // 4096, 1)
    dx, dw = B.f8_gemm_grad(x, w, dy)
    want = (dyb.double() @ dense(v, s)).to(BF).to(DEV)
    assert all(torch.equal(part, want) for part in dx.view(-1, 4096, k))
    assert torch.equal(dw.cpu(), ((dyb.double().T @ base.double()) * (m // 4096)).float())   # below 2^24


def test_experts_past_32_bits_of_bytes():
    E, n, k = 280, 4096, 4096
    few = torch.randint(-4, 5, (7, n, k), generator=gen(1)).float().to(E4M3).view(torch.uint8).to(DEV)
    v = few.repeat(E // 7, 1, 1)
    s = torch.full((E, n // 128, k // 128), 127, dtype=torch.uint8, device=DEV)
    w = B.f8_weight(v, s)
    del v
    one = [B.f8_weight(few[e], s[e]) for e in range(7)]
    for tokens in (4, 300):
        x = whole(tokens, k, 2, 1).to(DEV)
        idx = torch.randint(E - 9, E, (tokens, 2), generator=gen(3)).int().to(DEV)
        y = B.f8_moe_gemm(x, w, idx).view(tokens, 2, n)
        for e in range(7):
            mine = B.f8_gemm(x, one[e])
            for slot in range(2):
                at = idx[:, slot] % 7 == e
                assert torch.equal(y[:, slot][at], mine[at])


def test_one_pair_more_than_the_registers_hold():
    """32768 pairs stay in registers while they are sorted, more are read twice."""
    E, n, k = 50, 32, 32
    v, s = whole_w(E, n, k, 1)
    wd = dense(v, s)
    w = B.f8_weight(v.to(DEV), s.to(DEV))
    for pairs in (32767, 32768, 32769, 50001):
        x = whole(pairs, k, 2)
        idx = torch.randint(-1, E, (pairs, 1), generator=gen(pairs)).int()
        y = B.f8_moe_gemm(x.to(DEV), w, idx.to(DEV))
        pick = wd[idx.flatten().clamp(min=0).long()]
        want = torch.bmm(pick, x.double().unsqueeze(-1)).squeeze(-1)
        want[idx.flatten() < 0] = 0
        assert torch.equal(y.cpu(), want.float()), pairs
