"""GPU tests that moe_route and moe_route_grad without a rule are the plain router:
bit for bit what binade_moe_route and binade_moe_route_grad give, called here
through the ABI."""
import ctypes

import pytest
import torch

from decode_gemv_tensor_amd import binade as B

pytestmark = pytest.mark.gpu

DEV = "cuda"


def P(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k,renorm", [(1, 128, 8, True), (500, 128, 8, True), (300, 60, 4, False), (70, 256, 12, True),
                                          (33, 1024, 64, False), (4000, 64, 2, True)])
def test_the_plain_routers_bits(T, E, k, renorm, dtype):
    g = torch.Generator()
    g.manual_seed(T + E)
    x = (torch.randn(T, E, generator=g) * 2).to(dtype).to(DEV)
    valid = (torch.rand(T, generator=g) < 0.8).to(DEV) if T > 1 else None
    st = torch.cuda.current_stream().cuda_stream
    L = B.lib()
    code = B.BF16 if dtype == torch.bfloat16 else B.F32
    idx = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k, device=DEV)
    counts = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    ps, loss = torch.empty(E, device=DEV), torch.empty(1, device=DEV)
    ws = torch.empty(L.binade_moe_route_workspace_bytes(T, E), dtype=torch.uint8, device=DEV)
    assert L.binade_moe_route(P(x), code, E, T, E, k, int(renorm), P(valid), P(idx), P(w), P(counts), P(ps), P(loss),
                              P(ws), ws.numel(), st) == B.OK
    dw, one = torch.randn(T, k, generator=g).to(DEV), torch.ones(1, device=DEV)
    d = torch.empty_like(x)
    assert L.binade_moe_route_grad(P(x), code, E, T, E, k, int(renorm), P(idx), P(dw), P(counts), P(one), P(d), code,
                                   E, None, st) == B.OK
    for kw in ({}, dict(score="softmax", bias=None, groups=1, top_groups=1, scale=1.0)):
        r = B.moe_route(x, k, renormalize=renorm, valid=valid, **kw)
        for name, a, b in (("idx", r.idx, idx), ("weights", r.weights, w), ("counts", r.counts, counts),
                           ("prob_sum", r.prob_sum, ps), ("loss", r.loss, loss)):
            assert torch.equal(a, b), name
        kw.pop("top_groups", None)
        got = B.moe_route_grad(x, idx, dweights=dw, counts=counts, dloss=one, renormalize=renorm, out_dtype=dtype, **kw)
        assert torch.equal(got.view(torch.uint8), d.view(torch.uint8))


def test_calls_that_go_by_a_rule_do_not_take_that_path():
    """The workspaces' checks tell the two entries apart: one too small for the
    entry that runs is refused by its name."""
    x = torch.randn(40, 64, device=DEV)
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    for kw, name in (({}, "binade_moe_route "), ({"scale": 2.0}, "binade_moe_route_scored"),
                     ({"score": "sigmoid"}, "binade_moe_route_scored"),
                     ({"bias": torch.zeros(64, device=DEV)}, "binade_moe_route_scored"),
                     ({"groups": 4, "top_groups": 2}, "binade_moe_route_scored")):
        with pytest.raises(B.BinadeError) as e:
            B.moe_route(x, 4, workspace=small, **kw)
        assert name.strip() in str(e.value) and ("scored" in str(e.value)) == ("scored" in name), (kw, str(e.value))
