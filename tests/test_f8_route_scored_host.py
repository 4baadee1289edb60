"""CPU tests of what the 8-bit products and the router by scores refuse: bad
arguments come back as status codes or exceptions before any HIP call, and
sizes of planes and workspaces are closed forms."""
import ctypes

import pytest
import torch

from decode_gemv_tensor_amd import binade as B

P = ctypes.c_void_p
GOOD = P(4096)


def _desc(**kw):
    d = B.F8Desc(256, 96, 1, B.E8M0, 4096, 4096, 4096, 4096)
    for key, v in kw.items():
        setattr(d, key, v)
    return d


def _ref(d):
    return None if d is None else ctypes.byref(d)


def _gemm(d, x=GOOD, m=20, ldx=96, y=GOOD, ldy=256, dt=B.F32, ws=GOOD, nb=1 << 40):
    return B.lib().binade_f8_gemm(_ref(d), x, m, ldx, y, ldy, dt, ws, nb, None)


def _grad(d, x=GOOD, m=20, ldx=96, dy=GOOD, ld_dy=256, dx=GOOD, ld_dx=96, dw=GOOD, dt=B.F32, ws=GOOD,
          nb=1 << 40):
    return B.lib().binade_f8_gemm_grad(_ref(d), x, m, ldx, dy, ld_dy, dx, ld_dx, dw, dt, ws, nb, None)


def _moe(d, x=GOOD, ldx=96, per_slot=0, idx=GOOD, t=200, k=2, y=GOOD, ldy=256, dt=B.F32, ws=GOOD, nb=1 << 40):
    return B.lib().binade_f8_moe_gemm(_ref(d), x, ldx, per_slot, idx, t, k, y, ldy, dt, ws, nb, None, None)


@pytest.mark.parametrize("call", [_gemm, _grad, _moe], ids=["gemm", "grad", "moe"])
def test_descriptors_are_checked(call):
    assert call(None) == B.EINVAL
    for kw in ({"rows": 0}, {"cols": -32}, {"count": 0}, {"values": None}, {"scales": None},
               {"scale_dtype": B.BF16}, {"scale_dtype": 3}):
        assert call(_desc(**kw)) == B.EINVAL, kw
    for kw in ({"cols": 48}, {"rows": (1 << 22) + 1}, {"cols": (1 << 22) + 32}, {"count": 65536},
               {"values": 4104}, {"scales": 4100}):
        assert call(_desc(**kw)) == B.EUNSUPPORTED, kw


@pytest.mark.parametrize("call", [_gemm, _grad, _moe], ids=["gemm", "grad", "moe"])
def test_workspaces_are_checked(call):
    assert call(_desc(), nb=0) == B.ENOSPACE
    assert call(_desc(), ws=None) == B.ENOSPACE
    assert call(_desc(), ws=P(4104)) == B.EUNSUPPORTED
    need = {_gemm: B.lib().binade_f8_gemm_workspace_bytes(20, 256, 96, B.F32),
            _grad: B.lib().binade_f8_gemm_grad_workspace_bytes(20, 256, 96, 1, 1, B.F32),
            _moe: B.lib().binade_f8_moe_workspace_bytes(200, 2, 0, 1, 256, 96)}[call]
    assert need > 0 and call(_desc(), nb=need - 1) == B.ENOSPACE


def test_gemm_refusals():
    for kw in ({"m": -1}, {"dt": 2}, {"dt": -1}, {"x": None}, {"y": None}, {"ldx": 88}, {"ldy": 255}):
        assert _gemm(_desc(), **kw) == B.EINVAL, kw
    assert _gemm(_desc(count=2)) == B.EINVAL
    for kw in ({"ldx": 100}, {"x": P(4104)}, {"m": (1 << 22) + 1}, {"ldx": (1 << 24) + 8},
               {"ldy": (1 << 24) + 1}):
        assert _gemm(_desc(), **kw) == B.EUNSUPPORTED, kw
    assert _gemm(_desc(rows=1 << 22), m=1 << 22, ldy=1 << 22) == B.EUNSUPPORTED   # m * N
    assert _gemm(_desc(), m=0, x=None, y=None, ws=None, nb=0) == B.OK


def test_grad_refusals():
    for kw in ({"m": -1}, {"dt": 2}, {"dy": None}, {"x": None}, {"ld_dy": 255}, {"ld_dx": 95}, {"ldx": 95}):
        assert _grad(_desc(), **kw) == B.EINVAL, kw
    assert _grad(_desc(count=2)) == B.EINVAL
    for kw in ({"values_t": None}, {"scales_t": None}):
        assert _grad(_desc(**kw)) == B.EINVAL, kw
    for kw in ({"values_t": 4100}, {"scales_t": 4104}):
        assert _grad(_desc(**kw)) == B.EUNSUPPORTED, kw
    for kw in ({"ldx": 100}, {"x": P(4104)}, {"m": (1 << 22) + 1}, {"ld_dy": (1 << 24) + 1},
               {"ld_dx": (1 << 24) + 1}, {"ldx": (1 << 24) + 8}):
        assert _grad(_desc(), **kw) == B.EUNSUPPORTED, kw
    assert _grad(_desc(), dx=None, dw=None, x=None) == B.OK   # nothing to do


def test_experts_refusals():
    for kw in ({"t": -1}, {"k": 0}, {"k": 65}, {"dt": 2}, {"x": None}, {"idx": None}, {"y": None}, {"ldx": 88},
               {"ldy": 255}):
        assert _moe(_desc(count=4), **kw) == B.EINVAL, kw
    for kw in ({"ldx": 100}, {"x": P(4104)}, {"t": (1 << 24) + 1, "k": 1}, {"t": 1 << 23, "k": 3},
               {"ldx": (1 << 24) + 8}, {"ldy": (1 << 24) + 1}):
        assert _moe(_desc(count=4), **kw) == B.EUNSUPPORTED, kw
    assert _moe(_desc(count=4097)) == B.EUNSUPPORTED
    assert _moe(_desc(count=4), t=0, x=None, idx=None, y=None) == B.OK


def test_planes():
    L = B.lib()
    s = B.F8Sizes()
    assert L.binade_f8_sizes_of(300, 416, 5, B.E8M0, ctypes.byref(s)) == B.OK
    assert (s.values_bytes, s.scales_bytes) == (5 * 300 * 512, 5 * 3 * 4)
    assert (s.values_t_bytes, s.scales_t_bytes) == (5 * 416 * 384, 5 * 4 * 4)
    assert L.binade_f8_sizes_of(1, 32, 1, B.F32, ctypes.byref(s)) == B.OK
    assert (s.values_bytes, s.scales_bytes, s.values_t_bytes, s.scales_t_bytes) == (128, 16, 4096, 16)
    for a in ((0, 32, 1, B.E8M0), (1, 0, 1, B.E8M0), (1, 32, 0, B.E8M0), (1, 32, 1, B.BF16)):
        assert L.binade_f8_sizes_of(*a, ctypes.byref(s)) == B.EINVAL, a
    for a in ((1, 33, 1, B.E8M0), ((1 << 22) + 1, 32, 1, B.E8M0), (1, 32, 65536, B.F32)):
        assert L.binade_f8_sizes_of(*a, ctypes.byref(s)) == B.EUNSUPPORTED, a
    assert L.binade_f8_sizes_of(1, 32, 1, B.E8M0, None) == B.EINVAL


def test_pack_and_layout_refusals():
    L = B.lib()
    for d in (_desc(rows=0), _desc(values=None), _desc(scales_t=None)):
        assert L.binade_f8_pack(GOOD, ctypes.byref(d), None) == B.EINVAL
        assert L.binade_f8_layout(GOOD, GOOD, ctypes.byref(d), None) == B.EINVAL
    assert L.binade_f8_pack(None, ctypes.byref(_desc()), None) == B.EINVAL
    assert L.binade_f8_pack(GOOD, None, None) == B.EINVAL
    assert L.binade_f8_pack(GOOD, ctypes.byref(_desc(scale_dtype=B.F32)), None) == B.EINVAL
    assert L.binade_f8_layout(None, GOOD, ctypes.byref(_desc()), None) == B.EINVAL
    assert L.binade_f8_layout(GOOD, None, ctypes.byref(_desc()), None) == B.EINVAL
    assert L.binade_f8_pack(P(4104), ctypes.byref(_desc()), None) == B.EUNSUPPORTED
    assert L.binade_f8_layout(P(4104), GOOD, ctypes.byref(_desc()), None) == B.EUNSUPPORTED
    assert L.binade_f8_layout(GOOD, P(4098), ctypes.byref(_desc(scale_dtype=B.F32)), None) == B.EUNSUPPORTED


def test_workspace_sizes():
    L = B.lib()
    assert L.binade_f8_gemm_workspace_bytes(16, 512, 512, B.F32) == 0          # up to 16 rows: none
    assert L.binade_f8_gemm_workspace_bytes(0, 512, 512, B.F32) == 0
    # rows of whole tiles, two blocks together, and four codes
    one = 192 * 512 + 192 * 4
    assert L.binade_f8_gemm_workspace_bytes(17, 1, 512, B.BF16) == one         # four blocks: one part
    assert L.binade_f8_gemm_workspace_bytes((1 << 22) + 1, 512, 512, B.F32) == 0
    assert L.binade_f8_gemm_grad_workspace_bytes(0, 64, 64, 1, 1, B.F32) == 0
    assert L.binade_f8_gemm_grad_workspace_bytes(20, 64, 64, 0, 0, B.F32) == 0
    both = L.binade_f8_gemm_grad_workspace_bytes(20, 64, 64, 1, 1, B.F32)
    assert both == L.binade_f8_gemm_grad_workspace_bytes(20, 64, 64, 1, 0, B.F32) + \
        L.binade_f8_gemm_grad_workspace_bytes(20, 64, 64, 0, 1, B.F32)
    assert L.binade_f8_moe_workspace_bytes(32, 8, 0, 16, 512, 512) == 0        # up to 256 pairs: none
    assert L.binade_f8_moe_workspace_bytes(33, 8, 0, 16, 512, 512) > 0
    assert L.binade_f8_moe_workspace_bytes(33, 65, 0, 16, 512, 512) == 0
    assert L.binade_f8_moe_workspace_bytes(33, 8, 0, 4097, 512, 512) == 0
    assert L.binade_moe_route_scored_workspace_bytes(-1, 64) == 0
    assert L.binade_moe_route_scored_workspace_bytes(64, 1025) == 0
    assert L.binade_moe_route_scored_workspace_bytes(64, 64) > 0


def test_scored_router_refusals():
    L = B.lib()

    def route(logits=GOOD, dt=B.F32, ld=16, t=4, e=16, k=2, rule=None, idx=GOOD, w=GOOD, c=GOOD, ps=GOOD,
              loss=GOOD, ws=GOOD, nb=1 << 30, **kw):
        r = dict(score=1, renormalize=1, groups=4, top_groups=2, group_best=2, scale=1.0, bias=4096)
        r.update(kw)
        r = B.RouteRule(*r.values())
        return L.binade_moe_route_scored(logits, dt, ld, t, e, k, ctypes.byref(r), None, idx, w, c, ps, loss,
                                         ws, nb, None)

    inf = float("inf")
    for kw in ({"ld": 15}, {"t": -1}, {"e": 0}, {"e": 1028, "ld": 2000}, {"k": 0}, {"k": 17}, {"dt": 2},
               {"logits": None}, {"idx": None}, {"w": None}, {"c": None}, {"ps": None}, {"loss": None},
               {"score": 2}, {"score": -1}, {"groups": 0}, {"groups": 3}, {"groups": 128, "e": 256, "ld": 256},
               {"top_groups": 0}, {"top_groups": 5}, {"group_best": 0}, {"group_best": 3}, {"scale": inf},
               {"scale": float("nan")}, {"k": 9}):
        assert route(**kw) == B.EINVAL, kw
    assert L.binade_moe_route_scored(GOOD, 0, 16, 4, 16, 2, None, None, GOOD, GOOD, None, None, None, None, 0,
                                     None) == B.EINVAL
    assert route(nb=0) == B.ENOSPACE and route(ws=None) == B.ENOSPACE
    assert route(nb=L.binade_moe_route_scored_workspace_bytes(4, 16) - 1) == B.ENOSPACE
    assert route(ws=P(4104)) == B.EUNSUPPORTED
    assert route(t=0, logits=None, idx=None, w=None, c=None, ps=None, loss=None) == B.OK

    def grad(logits=GOOD, dt=B.F32, ld=16, t=4, e=16, k=2, score=1, scale=1.0, idx=GOOD, c=GOOD, dl=GOOD,
             out=GOOD, odt=B.F32, ldd=16):
        return L.binade_moe_route_scored_grad(logits, dt, ld, t, e, k, score, 1, scale, idx, GOOD, c, dl, out,
                                              odt, ldd, None, None)

    for kw in ({"ld": 15}, {"ldd": 15}, {"t": -1}, {"e": 0}, {"k": 0}, {"k": 17}, {"dt": 3}, {"odt": 3},
               {"score": 2}, {"scale": inf}, {"logits": None}, {"idx": None}, {"out": None}, {"c": None},
               {"dl": None}):
        assert grad(**kw) == B.EINVAL, kw
    assert grad(t=0) == B.OK


def test_bindings_check_before_calling():
    with pytest.raises(ValueError, match="device tensors"):
        B.f8_gemm(torch.zeros(1, 32, dtype=torch.bfloat16), None)
    with pytest.raises(ValueError, match="device tensors"):
        B.f8_pack(torch.zeros(1, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        B.moe_route(torch.zeros(1, 8), 2, score="sigmoid")
