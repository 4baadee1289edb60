"""CPU tests of the adapter and router entry points' refusals: bad arguments
come back as status codes or exceptions before any HIP call, and workspace
sizes are closed forms of the sizes."""
import ctypes
import os

import pytest
import torch

from decode_gemv_tensor_amd import binade as B

P = ctypes.c_void_p
GOOD = P(4096)


def _desc(**kw):
    d = B.LoraDesc()
    d.n, d.k, d.rank, d.n_adapters, d.a, d.b = 40, 64, 16, 3, 4096, 4096
    for key, v in kw.items():
        setattr(d, key, v)
    return d


def _add(d, x=GOOD, m=2, ldx=64, ids=GOOD, base=GOOD, ld_base=40, bdt=B.F32, y=GOOD, ldy=40,
         ydt=B.F32, h=None, ws=GOOD, nb=1 << 30):
    return B.lib().binade_lora_add(None if d is None else ctypes.byref(d), x, m, ldx, ids, base,
                                   ld_base, bdt, y, ldy, ydt, h, ws, nb, None, None)


def _grad(d, x=GOOD, m=2, ldx=64, ids=GOOD, dy=GOOD, ld_dy=40, h=None, dxb=GOOD, ld_dxb=64,
          dx=GOOD, ld_dx=64, da=GOOD, db=GOOD, gdt=B.F32, ws=GOOD, nb=1 << 30):
    return B.lib().binade_lora_grad(None if d is None else ctypes.byref(d), x, m, ldx, ids, dy,
                                    ld_dy, h, dxb, ld_dxb, dx, ld_dx, da, db, gdt, ws, nb, None,
                                    None)


@pytest.mark.parametrize("call", [_add, _grad], ids=["add", "grad"])
def test_lora_descriptor_and_input_refusals(call):
    assert call(None) == B.EINVAL
    for kw in ({"n": 0}, {"k": -64}, {"rank": 0}, {"n_adapters": 0}, {"a": None}, {"b": None}):
        assert call(_desc(**kw)) == B.EINVAL, kw
    for kw in ({"k": 48}, {"rank": 12}, {"rank": 136}, {"n_adapters": 65536}, {"a": 4104},
               {"b": 4098}):
        assert call(_desc(**kw), ldx=64) == B.EUNSUPPORTED, kw
    assert call(_desc(), m=-1) == B.EINVAL
    assert call(_desc(), x=None) == B.EINVAL
    assert call(_desc(), ldx=56) == B.EINVAL
    assert call(_desc(), ldx=68) == B.EUNSUPPORTED
    assert call(_desc(), ldx=(1 << 24) + 8) == B.EUNSUPPORTED
    assert call(_desc(), x=P(4104)) == B.EUNSUPPORTED
    assert call(_desc(), nb=0) == B.ENOSPACE
    assert call(_desc(), ws=None) == B.ENOSPACE
    assert call(_desc(), ws=P(4104)) == B.EUNSUPPORTED


def test_lora_add_refusals():
    assert _add(_desc(), y=None) == B.EINVAL
    assert _add(_desc(), ldy=39) == B.EINVAL
    assert _add(_desc(), ld_base=39) == B.EINVAL
    assert _add(_desc(), bdt=2) == B.EINVAL
    assert _add(_desc(), ydt=-1) == B.EINVAL
    assert _add(_desc(), m=0, x=None, y=None, ws=None, nb=0) == B.OK


def test_lora_grad_refusals():
    assert _grad(_desc(), dy=None) == B.EINVAL
    assert _grad(_desc(), ld_dy=39) == B.EINVAL
    assert _grad(_desc(), ld_dy=(1 << 24) + 1) == B.EUNSUPPORTED
    assert _grad(_desc(), da=None) == B.EINVAL
    assert _grad(_desc(), db=None) == B.EINVAL
    assert _grad(_desc(), gdt=5) == B.EINVAL
    assert _grad(_desc(), ld_dx=56) == B.EINVAL
    assert _grad(_desc(), ld_dxb=56) == B.EINVAL
    assert _grad(_desc(), ld_dx=68) == B.EUNSUPPORTED
    assert _grad(_desc(), ld_dxb=68) == B.EUNSUPPORTED
    assert _grad(_desc(), dx=P(4100)) == B.EUNSUPPORTED
    assert _grad(_desc(), dxb=P(4100)) == B.EUNSUPPORTED


def test_router_refusals():
    L = B.lib()

    def route(logits=GOOD, dt=B.F32, ld=16, t=4, e=16, k=2, idx=GOOD, w=GOOD, c=GOOD, ps=GOOD,
              loss=GOOD, ws=GOOD, nb=1 << 30):
        return L.binade_moe_route(logits, dt, ld, t, e, k, 1, None, idx, w, c, ps, loss, ws, nb,
                                  None)

    for kw in ({"ld": 15}, {"t": -1}, {"e": 0}, {"e": 1025, "ld": 2000}, {"k": 0}, {"k": 17},
               {"e": 128, "ld": 128, "k": 65}, {"dt": 2}, {"logits": None}, {"idx": None},
               {"w": None}, {"c": None}, {"ps": None}, {"loss": None}):
        assert route(**kw) == B.EINVAL, kw
    assert route(nb=0) == B.ENOSPACE and route(ws=None) == B.ENOSPACE
    assert route(ws=P(4104)) == B.EUNSUPPORTED
    assert route(t=0, logits=None, idx=None, w=None, c=None, ps=None, loss=None) == B.OK

    def grad(logits=GOOD, dt=B.F32, ld=16, t=4, e=16, k=2, idx=GOOD, c=GOOD, dl=GOOD, out=GOOD,
             odt=B.F32, ldd=16):
        return L.binade_moe_route_grad(logits, dt, ld, t, e, k, 1, idx, GOOD, c, dl, out, odt, ldd,
                                       None, None)

    for kw in ({"ld": 15}, {"ldd": 15}, {"t": -1}, {"e": 0}, {"k": 0}, {"k": 17}, {"dt": 3},
               {"odt": 3}, {"logits": None}, {"idx": None}, {"out": None}, {"c": None},
               {"dl": None}):
        assert grad(**kw) == B.EINVAL, kw
    assert grad(t=0) == B.OK


def test_combine_grad_refusals():
    L = B.lib()

    def grad(y=GOOD, w=GOOD, d=GOOD, ddt=B.F32, t=2, k=2, n=8, dy=GOOD, dt=B.F32, dw=GOOD):
        return L.binade_moe_combine_grad(y, w, d, ddt, t, k, n, dy, dt, dw, None)

    for kw in ({"y": None}, {"w": None}, {"d": None}, {"ddt": 2}, {"dt": 2}, {"t": -1}, {"k": 0},
               {"k": 65}, {"n": -1}, {"dw": None}):
        assert grad(**kw) == B.EINVAL, kw
    assert grad(t=0) == B.OK


def test_workspace_sizes():
    L = B.lib()
    for bad in ((-1, 40, 64, 16), (4, 0, 64, 16), (4, 40, 48, 16), (4, 40, 64, 12)):
        assert L.binade_lora_workspace_bytes(*bad) == 0
        assert L.binade_lora_grad_workspace_bytes(*bad, 2) == 0
    assert L.binade_lora_grad_workspace_bytes(4, 40, 64, 16, 0) == 0
    assert L.binade_moe_route_workspace_bytes(4, 0) == 0
    assert L.binade_moe_route_workspace_bytes(4, 1025) == 0
    assert L.binade_lora_workspace_bytes(4, 40, 64, 16) > 0
    assert L.binade_moe_route_workspace_bytes(0, 16) > 0


def test_bindings_refuse_host_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    a, b = torch.zeros(1, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 40, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.lora_add(x, a, b)
    with pytest.raises(ValueError):
        B.lora_grad(x, a, b, None, torch.zeros(2, 40, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        B.moe_route(torch.zeros(2, 16), 2)
    with pytest.raises(ValueError):
        B.moe_route_grad(torch.zeros(2, 16), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        B.moe_combine_grad(torch.zeros(4, 8), torch.zeros(2, 2), torch.zeros(2, 8), 2)


def test_lora_descriptor_matches_the_c_compiler(tmp_path):
    import subprocess
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    src = tmp_path / "s.c"
    src.write_text("""#include <stdio.h>
#include <stddef.h>
#include "binade.h"
int main(void) {
  printf("%zu %zu %zu %zu\\n", sizeof(binade_lora), offsetof(binade_lora, rank),
         offsetof(binade_lora, a), offsetof(binade_lora, scale));
  return 0;
}
""")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-std=c99", "-I", inc, str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(B.LoraDesc), B.LoraDesc.rank.offset, B.LoraDesc.a.offset,
                   B.LoraDesc.scale.offset]


def _router_blocks(tokens, experts, bf16):
    """Blocks of the router's kernel, each of which leaves a row of partial
    counts and sums. lanes: those of a token; a wave has 64 / lanes tokens."""
    lanes = 8 if experts <= 128 else 16 if experts <= 256 else 32 if experts <= 512 else 64
    if not bf16 and 64 < experts <= 512:
        lanes *= 2
    waves = -(-tokens * lanes // 64)
    a_block = 1 if waves <= 1 else 4 if waves <= 1024 else 16
    return max(1, min(256, -(-waves // a_block)))


@pytest.mark.parametrize("experts", [1, 64, 65, 128, 129, 256, 257, 512, 513, 1024])
def test_router_workspace_holds_the_blocks_of_both_types(experts):
    """More waves may mean fewer blocks (four waves a block up to 1024 waves,
    sixteen behind), so neither type's size covers the other's everywhere."""
    f = B.lib().binade_moe_route_workspace_bytes
    at = {0, 1 << 20, 1 << 30}
    for lanes in (8, 16, 32, 64):
        for waves in (1, 1024, 4096):       # the switches, and where the blocks are full
            at.update(range(max(0, waves * 64 // lanes - 70), waves * 64 // lanes + 70))
    at.update(range(0, 70000, 97))
    for tokens in sorted(at):
        blocks = max(_router_blocks(tokens, experts, bf16) for bf16 in (False, True))
        assert f(tokens, experts) >= 128 + 4 * blocks * (2 * experts + 1), tokens


def _one_row_views(k, dtype):
    """Single rows of k values that torch calls contiguous, at row strides
    that the calls do not take."""
    column = torch.arange(k, dtype=torch.float32).to(dtype).reshape(k, 1)
    wide = torch.zeros(3, k + 4, dtype=dtype)
    wide[:, :k] = column.t()
    far = torch.zeros((1 << 24) // k + 2, k, dtype=dtype)
    far[-1] = column[:, 0]
    return [column.t(), wide[:1, :k], far[None][:, -1], column.t().contiguous().expand(1, k)]


def test_a_single_rows_stride_is_of_no_matter():
    cpu = torch.device("cpu")
    for t in _one_row_views(64, torch.bfloat16):
        rows, ld = B._rows16("x", t, 64, cpu)
        assert ld == 64 and rows.data_ptr() % 16 == 0 and torch.equal(rows, t)
    for t in _one_row_views(64, torch.float32):
        rows, ld = B._logits_arg(t)
        assert ld == 64 and torch.equal(rows, t)
    off = torch.arange(72, dtype=torch.float32).to(torch.bfloat16)[1:65].as_strided((1, 64), (3, 1))
    rows, ld = B._rows16("x", off, 64, cpu)
    assert ld == 64 and rows.data_ptr() % 16 == 0 and torch.equal(rows, off)


def test_rows_at_strides_that_the_calls_do_not_take_are_copied():
    cpu = torch.device("cpu")
    big = torch.zeros(2 << 24, dtype=torch.bfloat16)
    for ld, copied in ((64, False), (72, False), (68, True), (0, True), (1 << 24, False),
                       ((1 << 24) + 8, True)):
        t = big.as_strided((2, 64), (ld, 1))
        rows, got = B._rows16("x", t, 64, cpu)
        assert (rows.data_ptr() != t.data_ptr()) == copied
        assert got == (64 if copied else ld)
    x = torch.arange(40, dtype=torch.float32)
    for t, ld in ((x.reshape(5, 8), 8), (x.reshape(5, 8)[:, :3], 8), (x.reshape(8, 5).t(), 8),
                  (x.as_strided((5, 8), (0, 1)), 8), (x[:5, None], 1), (x[:0].reshape(0, 8), 8)):
        rows, got = B._logits_arg(t)
        assert got == ld and torch.equal(rows, t)


def test_bindings_take_every_argument_by_name():
    """The first one too: host tensors get as far as the check for them."""
    x, z = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 16)
    a, b = torch.zeros(1, 8, 64, dtype=torch.bfloat16), torch.zeros(1, 40, 8, dtype=torch.bfloat16)
    for call, kw in ((B.lora_add, dict(x=x, a=a, b=b)),
                     (B.lora_grad, dict(b=b, a=a, x=x, ids=None, dy=x)),
                     (B.moe_route, dict(top_k=2, logits=z)),
                     (B.moe_route_grad, dict(logits=z, idx=z)),
                     (B.moe_combine_grad, dict(y=z, weights=z, dout=z, top_k=1))):
        with pytest.raises(ValueError, match="takes device tensors"):
            call(**kw)


def test_combine_grad_refuses_more_slots_than_it_counts():
    """Also where the product of tokens and slots does not fit 64 bits."""
    L = B.lib()
    for t, k, n in (((1 << 30) + 1, 1, 8), ((1 << 24) + 1, 64, 8), ((1 << 30) // 3 + 1, 3, 8),
                    (1 << 58, 64, 8), (1 << 62, 4, 8), ((1 << 63) - 1, 64, 8),
                    ((1 << 63) // 64 + 1, 64, 8), (2, 2, (1 << 30) + 1)):
        assert L.binade_moe_combine_grad(GOOD, GOOD, GOOD, B.F32, t, k, n, GOOD, B.F32, GOOD,
                                         None) == B.EUNSUPPORTED, (t, k, n)
