"""GPU tests of the low-rank adapters beside a shared projection
(binade_lora_add, binade_lora_grad) against their formulas in 64 bits.

Two kinds of inputs. Small whole numbers, for which every sum and product is
exact in fp32 (all magnitudes below 2^24) and in any order: results have to
be equal, bit for bit. Normal values, where an error is held to what fp32 sums
cost: a chain of L additions of terms of random sign has a relative error of
about u sqrt(L / 6), u = 2^-24 (the partial sum's rms grows as sqrt(j), each
addition rounds by u / sqrt(3) of it at most); three times that, summed over
the chains, is the tolerance of the 2-norm. A bf16 output adds half a step,
2^-8 of the value, per element."""
import ctypes
import math

import pytest
import torch

from decode_gemv_tensor_amd import binade as B

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def say(*a):
    print(*a, flush=True)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def make(m, n, k, rank, na, seed, whole=True, ids="mix"):
    g = gen(seed)

    def draw(*shape, hi=2, sigma=1.0):
        if whole:
            return torch.randint(-hi, hi + 1, shape, generator=g).to(BF)
        return (torch.randn(*shape, generator=g) * sigma).to(BF)

    x = draw(m, k)
    a = draw(na, rank, k, hi=1, sigma=k ** -0.5)
    b = draw(na, n, rank, hi=1, sigma=rank ** -0.5)
    if whole:
        scale = 2.0 ** torch.randint(-1, 2, (na,), generator=g).float()
        a = a * (torch.rand(na, rank, k, generator=g) < 24.0 / k).to(BF)   # keeps h small
    else:
        scale = torch.rand(na, generator=g) + 0.5
    base = draw(m, n, hi=9)
    dy = draw(m, n, hi=1, sigma=1e-2)
    if whole:
        dy = dy * (torch.rand(m, n, generator=g) < 24.0 / n).to(BF)
    if ids == "mix":
        i = torch.randint(-1, na, (m,), generator=g).to(torch.int32)
    elif ids == "runs":
        i = (torch.arange(m) * (na + 1) // max(m, 1) - 1).to(torch.int32)
    elif ids == "none":
        i = torch.full((m,), -1, dtype=torch.int32)
    else:
        i = None
    return {"x": x, "a": a, "b": b, "scale": scale, "base": base, "dy": dy, "ids": i}


def ref_add(d, scale=True, base=True):
    """In float64, worked out on the device, given back on the host."""
    m, na = d["x"].shape[0], d["a"].shape[0]
    ids = torch.zeros(m, dtype=torch.int32) if d["ids"] is None else d["ids"]
    x = d["x"].to(DEV).double()
    y = (d["base"].to(DEV).double().clone() if base
         else torch.zeros(m, d["b"].shape[1], dtype=torch.float64, device=DEV))
    h = torch.zeros(m, d["a"].shape[1], dtype=torch.float64, device=DEV)
    for i in range(na):
        t = (ids == i).nonzero()[:, 0].to(DEV)
        if not t.numel():
            continue
        h[t] = x[t] @ d["a"][i].to(DEV).double().T
        s = float(d["scale"][i]) if scale else 1.0
        y[t] += s * (h[t] @ d["b"][i].to(DEV).double().T)
    return y.cpu(), h.cpu()


def ref_grad(d, h, scale=True, base=None):
    m, k = d["x"].shape
    na, rank = d["a"].shape[:2]
    n = d["b"].shape[1]
    ids = torch.zeros(m, dtype=torch.int32) if d["ids"] is None else d["ids"]
    dx = (base.to(DEV).double().clone() if base is not None
          else torch.zeros(m, k, dtype=torch.float64, device=DEV))
    da = torch.zeros(na, rank, k, dtype=torch.float64, device=DEV)
    db = torch.zeros(na, n, rank, dtype=torch.float64, device=DEV)
    x, dy, h = d["x"].to(DEV).double(), d["dy"].to(DEV).double(), h.to(DEV)
    for i in range(na):
        t = (ids == i).nonzero()[:, 0].to(DEV)
        if not t.numel():
            continue
        s = float(d["scale"][i]) if scale else 1.0
        g = s * (dy[t] @ d["b"][i].to(DEV).double())
        dx[t] += g @ d["a"][i].to(DEV).double()
        da[i] = g.T @ x[t]
        db[i] = s * (dy[t].T @ h[t])
    return dx.cpu(), da.cpu(), db.cpu()


def to_dev(d):
    return {k: None if v is None else v.to(DEV) for k, v in d.items()}


def rel(x, ref):
    ref = ref.double()
    off = (x.double().cpu() - ref.cpu()).norm()
    return float(off / ref.norm()) if float(ref.norm()) else float(off)


def chain(n):
    return 3 * U * (math.sqrt(n / 6) + 1)


# the last dimension of a tile, a slice and a group on both sides of its end
ADD = [(1, 64, 64, 8, 1, "one"), (1, 1001, 96, 16, 3, "mix"), (2, 17, 32, 128, 5, "mix"),
       (15, 33, 256, 24, 2, "mix"), (16, 256, 1056, 32, 4, "runs"), (17, 515, 544, 16, 7, "mix"),
       (33, 1, 2080, 40, 3, "mix"), (64, 96, 512, 64, 2, "one"), (65, 1000, 4128, 8, 9, "runs"),
       (130, 130, 288, 56, 1, "mix"), (257, 264, 1024, 120, 33, "mix"), (300, 48, 64, 72, 64, "mix"),
       (1029, 72, 160, 16, 6, "runs"),
       # one launch for a few rows of one or two adapters
       (16, 300, 288, 32, 2, "mix"), (7, 1000, 4128, 24, 1, "mix"), (1, 130, 8192, 32, 4, "mix"),
       (2, 513, 96, 8, 9, "mix"),
       # running sums apart, many rows
       (520, 48, 2336, 16, 3, "mix"), (577, 6700, 96, 8, 3, "mix"), (600, 6661, 544, 40, 5, "runs"),
       (1030, 4200, 64, 72, 4, "mix"), (530, 7200, 288, 128, 2, "one"), (2051, 2050, 2080, 32, 6, "runs"),
       (5, 40, 128, 8, 3, "none"), (600, 6661, 64, 8, 3, "none"),
       (1500, 3001, 96, 16, 40, "mix"),
       # many rows for one adapter alone
       (130, 16500, 96, 16, 1, "mix"), (257, 8201, 160, 72, 3, "one")]


@pytest.mark.parametrize("case", ADD, ids=lambda c: "x".join(map(str, c)))
def test_add_is_exact_on_whole_numbers(case):
    m, n, k, rank, na, ids = case
    d = make(m, n, k, rank, na, seed=sum(case[:5]), ids=ids)
    y_ref, h_ref = ref_add(d)
    assert float(h_ref.abs().max()) < 2 ** 24 and float(y_ref.abs().max()) < 2 ** 22
    v = to_dev(d)
    for base_dt in (BF, F32):
        say("lora_add", case, base_dt)
        y, h = B.lora_add(v["x"], v["a"], v["b"], v["ids"], base=v["base"].to(base_dt),
                          scale=v["scale"], out_dtype=F32, keep_h=True)
        assert torch.equal(y.cpu().double(), y_ref)
        assert torch.equal(h.cpu().double(), h_ref)
        yb = B.lora_add(v["x"], v["a"], v["b"], v["ids"], base=v["base"].to(base_dt),
                        scale=v["scale"], out_dtype=BF)
        assert torch.equal(yb.cpu().float(), y_ref.float().to(BF).float())
    y = B.lora_add(v["x"], v["a"], v["b"], v["ids"])       # no base, no scale
    assert torch.equal(y.cpu().double(), ref_add(d, scale=False, base=False)[0])


@pytest.mark.parametrize("case", [c for c in ADD if c[5] != "none"], ids=lambda c: "x".join(map(str, c)))
def test_add_rounds_as_fp32_sums_do(case):
    m, n, k, rank, na, ids = case
    d = make(m, n, k, rank, na, seed=7 + sum(case[:5]), whole=False, ids=ids)
    y_ref, h_ref = ref_add(d, base=False)
    v = to_dev(d)
    y, h = B.lora_add(v["x"], v["a"], v["b"], v["ids"], scale=v["scale"], keep_h=True)
    say("lora_add", case, rel(h, h_ref), rel(y, y_ref))
    assert rel(h, h_ref) <= chain(k)
    assert rel(y, y_ref) <= chain(k) + chain(3 * rank)
    y_ref, _ = ref_add(d)
    yb = B.lora_add(v["x"], v["a"], v["b"], v["ids"], base=v["base"], scale=v["scale"],
                    out_dtype=BF).cpu().double()
    # half a bf16 step, and the fp32 sums' error against the largest value of the row
    tol = 2.0 ** -8 * y_ref.abs() + 8 * (chain(k) + chain(3 * rank)) * y_ref.abs().amax(1, True)
    assert bool(((yb - y_ref).abs() <= tol).all())


@pytest.mark.parametrize("size", [(150, 264, 2080, 24), (600, 6700, 2336, 24), (150, 264, 96, 16)],
                         ids=lambda c: "x".join(map(str, c)))
def test_a_row_does_not_depend_on_the_others(size):
    m, n, k, rank = size
    na = 5
    d = to_dev(make(m, n, k, rank, na, seed=3, whole=False))
    y, h = B.lora_add(d["x"], d["a"], d["b"], d["ids"], base=d["base"], scale=d["scale"],
                      keep_h=True)
    perm = torch.randperm(m, generator=gen(1)).to(DEV)
    for t in [perm, perm[:70], perm[:17], perm[:16], perm[3:4], perm[3:5]]:
        say("rows", t.numel())
        y2, h2 = B.lora_add(d["x"][t], d["a"], d["b"], d["ids"][t], base=d["base"][t],
                            scale=d["scale"], keep_h=True)
        assert torch.equal(y2, y[t]) and torch.equal(h2, h[t])
    # many rows, all of one adapter, against the same rows among the others
    one = (d["ids"] == 2).nonzero()[:, 0]
    for t in (one.repeat(1000 // one.numel() + 1), one[:9]):
        y2 = B.lora_add(d["x"][t], d["a"][2:3], d["b"][2:3], None, base=d["base"][t],
                        scale=d["scale"][2:3])
        assert torch.equal(y2, y[t])


@pytest.mark.parametrize("size", [(70, 136, 544, 16), (640, 6700, 288, 24), (1100, 64, 4224, 40),
                                  (2200, 15400, 96, 16)],
                         ids=lambda c: "x".join(map(str, c)))
def test_nan_and_infinity_stay_in_their_rows_and_adapters(size):
    m, n, k, rank = size
    na = 4
    d = make(m, n, k, rank, na, seed=11)
    d["ids"][[4, 9, 13]] = torch.tensor([0, 0, 2], dtype=torch.int32)
    clean = to_dev(d)
    y0 = B.lora_add(clean["x"], clean["a"], clean["b"], clean["ids"], base=clean["base"])
    h0 = ref_add(d, scale=False)[1]
    g0 = B.lora_grad(clean["x"], clean["a"], clean["b"], clean["ids"], clean["dy"])
    d["a"][1, 3, 5] = float("nan")
    d["b"][1, 7, 2] = float("inf")
    d["x"][4] = float("nan")
    d["x"][9, 8] = float("-inf")
    d["base"][11, 0] = float("inf")
    d["dy"][13] = float("nan")
    v = to_dev(d)
    y = B.lora_add(v["x"], v["a"], v["b"], v["ids"], base=v["base"])
    fine = torch.ones(m, dtype=torch.bool)
    fine[[4, 9, 11, 13]] = False
    fine &= d["ids"] != 1
    assert torch.equal(y.cpu()[fine], y0.cpu()[fine])
    assert bool(torch.isnan(y[4]).all())
    dx, da, db = B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"], h=h0.float().to(DEV))
    fine[[4, 9]] = True               # neither x nor base reaches dx
    fine[11] = int(d["ids"][11]) != 1
    assert torch.equal(dx.cpu()[fine], g0[0].cpu()[fine])
    assert torch.equal(da[3], g0[1][3]) and torch.equal(db[3], g0[2][3])
    assert bool(torch.isnan(dx[13]).all()) and bool(torch.isnan(db[2]).any())


def test_bad_ids_are_flagged_and_count_as_none():
    d = make(40, 72, 96, 16, 3, seed=5)
    d["ids"][[0, 7, 39]] = torch.tensor([3, -2, 2 ** 31 - 1], dtype=torch.int32)
    none = dict(d, ids=d["ids"].clone())
    none["ids"][[0, 7, 39]] = -1
    v = to_dev(d)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y, h = B.lora_add(v["x"], v["a"], v["b"], v["ids"], base=v["base"], keep_h=True, status=status)
    assert int(status.item()) == B.DEV_BAD_INDEX
    y_ref, h_ref = ref_add(none, scale=False)
    assert torch.equal(y.cpu().double(), y_ref) and torch.equal(h.cpu().double(), h_ref)
    status.zero_()
    got = B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"], status=status)
    assert int(status.item()) == B.DEV_BAD_INDEX
    for x, r in zip(got, ref_grad(none, h_ref, scale=False)):
        assert torch.equal(x.cpu().double(), r.to(x.dtype).double())
    status.zero_()
    w = none["ids"].to(DEV)
    B.lora_add(v["x"], v["a"], v["b"], w, status=status)
    B.lora_grad(v["x"], v["a"], v["b"], w, v["dy"], status=status)
    assert int(status.item()) == 0


def test_strides_in_place_and_rows_behind_the_last():
    m, n, k, rank, na = 21, 43, 160, 16, 3
    d = make(m, n, k, rank, na, seed=8)
    v = to_dev(d)
    y_ref, h_ref = ref_add(d)
    wide = torch.full((m + 2, k + 24), 7.0, dtype=BF, device=DEV)
    wide[:m, :k] = v["x"]
    assert torch.equal(B.lora_add(wide[:m, :k], v["a"], v["b"], v["ids"], base=v["base"],
                                  scale=v["scale"]).cpu().double(), y_ref)
    base = v["base"].float()
    assert B.lora_add(v["x"], v["a"], v["b"], v["ids"], base=base, scale=v["scale"], y=base) is base
    assert torch.equal(base.cpu().double(), y_ref)
    # through the C ABI: output rows at an odd stride, gaps and rows behind m left alone
    desc, keep = B._lora_desc(v["a"], v["b"], v["scale"], v["x"].device)[:2]
    ws = torch.empty(B.lib().binade_lora_workspace_bytes(m, n, k, rank), dtype=torch.uint8,
                     device=DEV)
    for dt, code in ((F32, B.F32), (BF, B.BF16)):
        y = torch.full((m + 3, n + 5), 99.0, dtype=dt, device=DEV)
        y[:m, :n] = v["base"]
        s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert B.lib().binade_lora_add(ctypes.byref(desc), B._ptr(wide), m, k + 24, B._ptr(v["ids"]),
                                       B._ptr(y), n + 5, code, B._ptr(y), n + 5, code, None,
                                       B._ptr(ws), ws.numel(), None, s) == B.OK
        torch.cuda.synchronize()
        assert torch.equal(y[:m, :n].cpu().double(), y_ref.to(dt).double())
        assert bool((y[m:] == 99).all()) and bool((y[:, n:] == 99).all())
    dx_ref, da_ref, db_ref = ref_grad(d, h_ref, base=d["x"])
    dyw = torch.full((m, n + 5), float("nan"), dtype=BF, device=DEV)
    dyw[:, :n] = v["dy"]
    dx = torch.full((m + 2, k + 8), 99.0, dtype=BF, device=DEV)
    dx[:m, :k] = v["x"]
    da = torch.empty(na, rank, k, device=DEV)
    db = torch.empty(na, n, rank, device=DEV)
    ws = torch.empty(B.lib().binade_lora_grad_workspace_bytes(m, n, k, rank, na),
                     dtype=torch.uint8, device=DEV)
    assert B.lib().binade_lora_grad(ctypes.byref(desc), B._ptr(wide), m, k + 24, B._ptr(v["ids"]),
                                    B._ptr(dyw), n + 5, None, B._ptr(dx), k + 8, B._ptr(dx), k + 8,
                                    B._ptr(da), B._ptr(db), B.F32, B._ptr(ws), ws.numel(), None,
                                    s) == B.OK
    torch.cuda.synchronize()
    assert torch.equal(dx[:m, :k].cpu().double(), dx_ref.to(BF).double())
    assert bool((dx[m:] == 99).all()) and bool((dx[:, k:] == 99).all())
    assert torch.equal(da.cpu().double(), da_ref) and torch.equal(db.cpu().double(), db_ref)


GRAD = [(1, 64, 64, 8, 1, "one"), (1, 33, 96, 16, 2, "mix"), (16, 128, 128, 16, 1, "one"),
        (31, 17, 32, 128, 3, "mix"), (32, 256, 1056, 32, 4, "runs"), (33, 515, 544, 24, 7, "mix"),
        (64, 1, 288, 40, 2, "mix"), (100, 130, 2080, 8, 5, "runs"), (257, 264, 512, 64, 9, "mix"),
        (513, 72, 160, 120, 2, "runs"), (1029, 200, 96, 16, 40, "mix"), (7, 40, 64, 8, 3, "none"),
        (2100, 136, 64, 16, 1, "one"),
        # running sums apart, many rows of dx, ranges of tiles over adapters
        (520, 2337, 64, 16, 3, "mix"), (577, 130, 6720, 16, 3, "mix"), (1030, 33, 4224, 72, 5, "runs"),
        (3001, 130, 288, 40, 9, "mix"), (2700, 72, 160, 120, 5, "runs"),
        (2051, 5, 2080, 24, 3, "runs"), (1500, 520, 96, 64, 1, "one"), (3000, 300, 64, 16, 200, "mix"),
        # dy read once for dB and g
        (34000, 1001, 32, 8, 1, "one"), (200, 64, 16416, 8, 1, "mix"), (4100, 8321, 64, 16, 200, "mix"), (2200, 15400, 96, 16, 3, "mix"),
        (8300, 4100, 4128, 16, 6, "runs")]


@pytest.mark.parametrize("case", GRAD, ids=lambda c: "x".join(map(str, c)))
def test_grad_is_exact_on_whole_numbers(case):
    m, n, k, rank, na, ids = case
    d = make(m, n, k, rank, na, seed=2 * sum(case[:5]), ids=ids)
    _, h_ref = ref_add(d)
    ref = ref_grad(d, h_ref, base=d["x"])
    assert all(float(r.abs().max()) < 2 ** 22 for r in ref)
    v = to_dev(d)
    for dt, h in ((F32, None), (BF, h_ref.float().to(DEV))):
        say("lora_grad", case, dt)
        dx, da, db = B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"], h=h, scale=v["scale"],
                                 dx_base=v["x"], grad_dtype=dt)
        assert torch.equal(dx.cpu().double(), ref[0].to(BF).double())
        assert torch.equal(da.cpu().double(), ref[1].to(dt).double())
        assert torch.equal(db.cpu().double(), ref[2].to(dt).double())
    # no scale, nothing upstream, nothing below
    ref = ref_grad(d, h_ref, scale=False)
    dx, da, db = B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"])
    assert torch.equal(dx.cpu().double(), ref[0].to(BF).double())
    none, da2, db2 = B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"], need_dx=False)
    assert none is None and torch.equal(da2, da) and torch.equal(db2, db)
    assert torch.equal(da.cpu().double(), ref[1]) and torch.equal(db.cpu().double(), ref[2])


@pytest.mark.parametrize("case", [c for c in GRAD if c[5] != "none"],
                         ids=lambda c: "x".join(map(str, c)))
def test_grad_rounds_as_fp32_sums_do(case):
    m, n, k, rank, na, ids = case
    d = make(m, n, k, rank, na, seed=5 + sum(case[:5]), whole=False, ids=ids)
    _, h_ref = ref_add(d)
    ref = ref_grad(d, h_ref)
    v = to_dev(d)
    dx, da, db = B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"], scale=v["scale"])
    say("lora_grad", case, rel(da, ref[1]), rel(db, ref[2]))
    # the sums over n (or k) and over the rows; h and g enter the second product as they are
    assert rel(da, ref[1]) <= chain(n) + chain(3 * m)
    assert rel(db, ref[2]) <= chain(k) + chain(3 * m)
    tol = 2.0 ** -8 * ref[0].abs() + 8 * (chain(n) + chain(3 * rank)) * ref[0].abs().amax(1, True)
    assert bool(((dx.cpu().double() - ref[0]).abs() <= tol).all())
    again = B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"], scale=v["scale"])
    assert all(torch.equal(p, q) for p, q in zip((dx, da, db), again))


def test_grad_is_the_difference_of_the_forward():
    """sum(dy * y) is linear in x, in a and in b: on whole numbers its exact
    difference along a direction is the gradient's product with it."""
    m, n, k, rank, na = 48, 96, 128, 16, 3
    d = make(m, n, k, rank, na, seed=21)
    v = to_dev(d)
    dx, da, db = B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"], scale=v["scale"])

    def f(**kw):
        w = dict(v, **kw)
        y = B.lora_add(w["x"], w["a"], w["b"], w["ids"], scale=w["scale"])
        return float((y.double() * v["dy"].double()).sum())

    f0, g = f(), gen(2)
    for name, grad in (("x", dx), ("a", da), ("b", db)):
        e = torch.randint(-1, 2, v[name].shape, generator=g).to(DEV)
        want = float((grad.double() * e).sum())
        assert want != 0
        assert f(**{name: v[name] + e.to(BF)}) - f0 == want


def test_no_rows():
    d = to_dev(make(0, 40, 64, 8, 2, seed=1))
    y, h = B.lora_add(d["x"], d["a"], d["b"], d["ids"], keep_h=True)
    assert y.shape == (0, 40) and h.shape == (0, 8)
    dx, da, db = B.lora_grad(d["x"], d["a"], d["b"], d["ids"], d["dy"])
    assert dx.shape == (0, 64) and not bool(da.any()) and not bool(db.any())
    assert da.shape == (2, 8, 64) and db.shape == (2, 40, 8)


def test_offsets_beyond_32_bits():
    """m * n over 2^31 elements (forward) and over 2^31 in dy (backward)."""
    n, k, rank = 32776, 64, 8
    m = 2 ** 31 // n + 40
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randint(-2, 3, (m, k), generator=g, device=DEV).to(BF)
    a = torch.randint(-1, 2, (2, rank, k), generator=g, device=DEV).to(BF)
    b = torch.randint(-1, 2, (2, n, rank), generator=g, device=DEV).to(BF)
    ids = torch.randint(-1, 2, (m,), generator=g, device=DEV).to(torch.int32)
    y = B.lora_add(x, a, b, ids, out_dtype=BF)
    tail = slice(m - 50, m)
    d = {"x": x[tail].cpu(), "a": a.cpu(), "b": b.cpu(), "ids": ids[tail].cpu(),
         "base": torch.zeros(50, n)}
    assert torch.equal(y[tail].cpu().double(), ref_add(d, scale=False)[0].to(BF).double())
    y.zero_()
    at = torch.randint(0, n, (m,), generator=g, device=DEV)
    y[torch.arange(m, device=DEV), at] = 1                     # dy: a one in each row
    dx, da, db = B.lora_grad(x, a, b, ids, y)
    d["dy"] = y[tail].cpu()
    h = ref_add(d, scale=False)[1]
    assert torch.equal(dx[tail].cpu().double(), ref_grad(d, h, scale=False)[0])
    hb = torch.zeros(2, n, rank, dtype=torch.float64, device=DEV)
    hx = torch.zeros(m, rank, dtype=torch.float64, device=DEV)
    for i in range(2):
        t = (ids == i).nonzero()[:, 0]
        hx[t] = x[t].double() @ a[i].double().T
        hb[i].index_add_(0, at[t], hx[t])
    assert torch.equal(db.double(), hb)


@pytest.mark.parametrize("size", [(40, 136, 544, 16), (2, 136, 544, 16), (1100, 4200, 96, 16),
                                  (2200, 15400, 96, 16)],
                         ids=lambda c: "x".join(map(str, c)))
def test_streams_and_graphs(size):
    m, n, k, rank = size
    na = 3
    cases = [to_dev(make(m, n, k, rank, na, seed=s, whole=False)) for s in (31, 32, 33)]
    want = []
    for v in cases:
        y, h = B.lora_add(v["x"], v["a"], v["b"], v["ids"], base=v["base"], scale=v["scale"],
                          keep_h=True)
        want.append((y, h) + B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"], h=h,
                                         scale=v["scale"], dx_base=v["x"]))
    torch.cuda.synchronize()
    # two calls at once on two streams, each with its own workspace
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for s, v in zip(streams, cases):
            y, h = B.lora_add(v["x"], v["a"], v["b"], v["ids"], base=v["base"], scale=v["scale"],
                              keep_h=True, stream=s)
            got.append((y, h) + B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"], h=h,
                                            scale=v["scale"], dx_base=v["x"], stream=s))
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert all(torch.equal(i, j) for i, j in zip(p, q))
    # captured once, replayed on other contents
    buf = {key: t.clone() for key, t in cases[0].items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = B.lora_add(buf["x"], buf["a"], buf["b"], buf["ids"], base=buf["base"],
                          scale=buf["scale"], keep_h=True)
        out = (y, h) + B.lora_grad(buf["x"], buf["a"], buf["b"], buf["ids"], buf["dy"], h=h,
                                   scale=buf["scale"], dx_base=buf["x"])
    for j in (1, 2, 0, 1, 2):
        for key, t in cases[j].items():
            buf[key].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want[j]))
        v = cases[j]
        B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"])      # eager work between replays


def test_a_workspace_of_the_size_asked_for_holds_it_all():
    """The caller's workspace, exactly as large as asked for, inside a larger
    buffer whose other bytes stay."""
    for m, n, k, rank, na in [(1, 64, 64, 8, 2), (45, 142, 96, 16, 12), (520, 2337, 64, 16, 3),
                              (600, 6700, 96, 40, 5), (300, 8000, 96, 24, 1), (2100, 3, 2080, 128, 7),
                              (2200, 15400, 96, 16, 5)]:
        d = make(m, n, k, rank, na, seed=m)
        v = to_dev(d)
        _, h_ref = ref_add(d, scale=False)
        for need, call in [
                (B.lib().binade_lora_workspace_bytes(m, n, k, rank),
                 lambda w: B.lora_add(v["x"], v["a"], v["b"], v["ids"], keep_h=True, workspace=w)),
                (B.lib().binade_lora_grad_workspace_bytes(m, n, k, rank, na),
                 lambda w: B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"], workspace=w))]:
            pool = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=DEV)
            assert pool.data_ptr() % 256 == 0
            got = call(pool[256:256 + need])
            want = call(None)
            assert bool((pool[:256] == 0xFF).all()) and bool((pool[256 + need:] == 0xFF).all())
            assert all(torch.equal(p, q) for p, q in zip(got, want))
            assert torch.isfinite(got[0]).all()
            if need == 0:          # one row of a small A needs none
                assert m == 1
                continue
            with pytest.raises(B.BinadeError) as e:
                call(pool[256:256 + need - 1])
            assert e.value.code == B.ENOSPACE


def test_beside_the_packed_products():
    """Decode (r4_gemv_rows) and prompt (r4_gemm) products with adapters in
    place, and the training pass with the projection's own input gradient."""
    g = gen(4)
    n, k, rank, na = 200, 256, 16, 4
    w = (torch.randn(n, k, generator=g) * 0.02).to(BF)
    r4 = B.rice_to_r4(B.pack_rice(w).to(DEV))
    for m in (1, 5, 8, 70):
        d = make(m, n, k, rank, na, seed=m, whole=False)
        v = to_dev(d)
        base = B.r4_gemv_rows(r4, v["x"]) if m <= 8 else B.r4_gemm(r4, v["x"])
        ref = ref_add(dict(d, base=d["x"].double() @ w.double().T))[0]
        y, h = B.lora_add(v["x"], v["a"], v["b"], v["ids"], base=base, scale=v["scale"], y=base,
                          keep_h=True)
        assert y is base
        assert rel(y, ref) <= 2 * chain(k) + chain(3 * rank)
        up = (v["dy"].double() @ B.unpack(r4).double()).to(BF)
        dx, da, db = B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"], h=h, scale=v["scale"],
                                 dx_base=up)
        rx, ra, rb = ref_grad(d, ref_add(d)[1], base=up.cpu())
        assert rel(da, ra) <= chain(n) + chain(3 * m) and rel(db, rb) <= chain(k) + chain(3 * m)
        assert rel(dx, rx) <= 2.0 ** -8


def test_one_row_at_any_stride():
    """A single row's stride is of no matter, whatever torch says it is."""
    k, n, rank = 64, 72, 8
    d = make(1, n, k, rank, 2, seed=6, ids="one")
    v = to_dev(d)
    want = B.lora_add(v["x"], v["a"], v["b"], None, base=v["base"])
    grads = B.lora_grad(v["x"], v["a"], v["b"], None, v["dy"], dx_base=v["x"])
    wide = torch.zeros(3, k + 4, dtype=BF, device=DEV)
    wide[:1, :k] = v["x"]
    far = torch.zeros(1, (1 << 24) // k + 2, k, dtype=BF, device=DEV)
    far[:, -1] = v["x"]
    for x in (v["x"].reshape(k, 1).t(), wide[:1, :k], far[:, -1]):
        say("one row", x.stride())
        assert torch.equal(B.lora_add(x, v["a"], v["b"], None, base=v["base"]), want)
        got = B.lora_grad(x, v["a"], v["b"], None, v["dy"], dx_base=x)
        assert all(torch.equal(p, q) for p, q in zip(got, grads))
        # of the other operands
        got = B.lora_grad(v["x"], v["a"], v["b"], None, v["dy"].reshape(n, 1).t(), dx_base=v["x"])
        assert all(torch.equal(p, q) for p, q in zip(got, grads))
        assert torch.equal(B.lora_add(v["x"], v["a"], v["b"], None,
                                      base=v["base"].reshape(n, 1).t()), want)


def test_arguments_by_name():
    v = to_dev(make(5, 40, 64, 8, 2, seed=2))
    y, h = B.lora_add(v["x"], v["a"], v["b"], v["ids"], keep_h=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for kw in ({}, {"stream": s}, {"stream": s.cuda_stream}):
        got = B.lora_add(a=v["a"], b=v["b"], x=v["x"], ids=v["ids"], keep_h=True, **kw)
        torch.cuda.synchronize()
        assert torch.equal(got[0], y) and torch.equal(got[1], h)


def test_the_most_rows_of_the_fewest_columns():
    """2^24 rows beside a projection of one output, several adapters in a
    tile: as many blocks of the first product as there can be."""
    m, n, k, rank, na = 1 << 24, 1, 1824, 8, 8
    g = gen(14)
    x = torch.zeros(m, k, dtype=BF, device=DEV)            # 61 GB
    a = torch.randint(-1, 2, (na, rank, k), generator=g).to(BF).to(DEV)
    b = torch.randint(-1, 2, (na, n, rank), generator=g).to(BF).to(DEV)
    ids = torch.full((m,), -1, dtype=torch.int32)
    rows = torch.cat([torch.arange(0, 40), torch.randint(0, m, (500,), generator=g),
                      torch.arange(m - 40, m)]).unique()
    ids[rows] = torch.randint(0, na, (rows.numel(),), generator=g).to(torch.int32)
    some = torch.randint(-1, 2, (rows.numel(), k), generator=g).to(BF)
    x[rows.to(DEV)] = some.to(DEV)
    y = B.lora_add(x, a, b, ids.to(DEV))
    del x
    torch.cuda.empty_cache()
    d = {"x": some, "a": a.cpu(), "b": b.cpu(), "ids": ids[rows], "base": torch.zeros(rows.numel(), n)}
    want = torch.zeros(m, n)
    want[rows] = ref_add(d, scale=False)[0].float()
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("m", [40, 3000])
def test_an_adapter_without_rows_gets_zeros_whatever_its_scale(m):
    """Gradients by adapter (few rows) and by ranges of rows (many)."""
    d = make(m, 72, 96, 16, 5, seed=m)
    d["ids"][d["ids"] == 2] = -1
    d["ids"][d["ids"] == 4] = 0
    v = to_dev(d)
    want = B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"], scale=v["scale"])
    v["scale"][2], v["scale"][4] = math.inf, math.nan
    for dt in (F32, BF):
        _, da, db = B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"], scale=v["scale"],
                                grad_dtype=dt)
        assert not bool(da[[2, 4]].any()) and not bool(db[[2, 4]].any())
        assert torch.equal(da, want[1].to(dt)) and torch.equal(db, want[2].to(dt))
    # no ids: adapter 0 alone has rows
    v["scale"][1] = -math.inf
    _, da, db = B.lora_grad(v["x"], v["a"], v["b"], None, v["dy"], scale=v["scale"])
    assert not bool(da[1:].any()) and not bool(db[1:].any()) and bool(db[0].any())


@pytest.mark.parametrize("rank", [8, 16, 24])
@pytest.mark.parametrize("m,n,k", [(2200, 15400, 960), (2200, 15400, 64), (2200, 300, 960),
                                   (20, 72, 64)])
def test_an_infinite_gradient_gives_an_infinite_input_gradient(m, n, k, rank):
    """Positive weights: g and dx of the row are +inf; ranks behind the last
    (8 of 16, 24 of 32) add nothing to it."""
    d = make(m, n, k, rank, 1, seed=rank, ids="one")
    d["a"][:], d["b"][:] = 1.0, 1.0
    v = to_dev(d)
    want = B.lora_grad(v["x"], v["a"], v["b"], None, v["dy"])[0]
    v["dy"][5, 3] = math.inf
    dx = B.lora_grad(v["x"], v["a"], v["b"], None, v["dy"])[0]
    assert bool((dx[5] == math.inf).all())
    fine = torch.arange(m) != 5
    assert torch.equal(dx[fine], want[fine])


def same(got, ref):
    """Equal, NaN where the reference has it and nowhere else."""
    got, ref = got.cpu(), ref.to(got.dtype)
    nan = torch.isnan(ref)
    return torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], ref[~nan])


@pytest.mark.parametrize("case", [(1, 64, 64, 8, 1, "one"), (16, 300, 288, 32, 2, "mix"),
                                  (33, 515, 544, 24, 7, "mix"), (65, 1000, 4128, 8, 9, "runs"),
                                  (257, 264, 1024, 120, 33, "mix"), (577, 6700, 96, 8, 3, "mix"),
                                  (600, 6661, 544, 40, 5, "runs"), (1030, 4200, 64, 72, 4, "mix"),
                                  (530, 7200, 288, 128, 2, "one"), (300, 8000, 96, 24, 1, "mix")],
                         ids=lambda c: "x".join(map(str, c)))
def test_infinite_weights_give_what_the_formula_gives(case):
    """h holds whole numbers, whose lower bf16 terms are 0: an infinite B
    beside them gives infinity (NaN only where h is 0), a NaN stays one. The
    same for A through h."""
    m, n, k, rank, na, ids = case
    d = make(m, n, k, rank, na, seed=3 * sum(case[:5]), ids=ids)
    i = int(d["ids"].max()) if d["ids"] is not None else 0
    i = max(i, 0)
    d["b"][i, n // 3, 2] = math.inf
    d["b"][i, n - 1, rank - 1] = -math.inf
    d["b"][i, 0, 1] = math.nan
    v = to_dev(d)
    y_ref, h_ref = ref_add(d)
    assert bool(torch.isinf(y_ref).any()) or m == 1
    for base_dt, dt in ((BF, F32), (F32, BF)):
        say("infinite b", case, base_dt)
        y, h = B.lora_add(v["x"], v["a"], v["b"], v["ids"], base=v["base"].to(base_dt),
                          scale=v["scale"], out_dtype=dt, keep_h=True)
        assert same(y, y_ref) and same(h, h_ref)
    d["a"][i, 3, k // 2] = math.inf
    d["x"][m // 2, 5] = -math.inf
    v = to_dev(d)
    y_ref, h_ref = ref_add(d)
    y, h = B.lora_add(v["x"], v["a"], v["b"], v["ids"], base=v["base"], scale=v["scale"],
                      keep_h=True)
    assert same(h, h_ref) and same(y, y_ref)


@pytest.mark.parametrize("case", [(1, 64, 64, 8, 1, "one"), (33, 515, 544, 24, 7, "mix"),
                                  (100, 130, 2080, 8, 5, "runs"), (577, 130, 6720, 16, 3, "mix"),
                                  (2051, 5, 2080, 24, 3, "runs"), (2100, 136, 64, 16, 1, "one"),
                                  (3001, 130, 288, 40, 9, "mix"), (1030, 33, 4224, 72, 5, "runs"),
                                  (34000, 1001, 32, 8, 1, "one"), (2200, 15400, 96, 16, 3, "mix"),
                                  (8300, 4100, 4128, 16, 6, "runs")],
                         ids=lambda c: "x".join(map(str, c)))
def test_infinite_operands_of_the_gradients_give_what_the_formulas_give(case):
    m, n, k, rank, na, ids = case
    d = make(m, n, k, rank, na, seed=5 * sum(case[:5]), ids=ids)
    _, h = ref_add(d)
    rows = torch.arange(m) if d["ids"] is None else (d["ids"] >= 0).nonzero()[:, 0]
    at = lambda f: int(rows[min(len(rows) - 1, int(f * len(rows)))])
    clean = d
    for name, r, c, val in (("x", at(0.3), k - 1, math.inf), ("x", at(0.99), 0, -math.inf),
                            ("dy", at(0.6), n - 1, math.inf), ("dy", at(0.1), n // 2, math.nan),
                            ("a", rank - 1, k // 2, -math.inf), ("x", at(0.5), None, math.inf)):
        say("infinite", name, case)
        d = dict(clean, **{name: clean[name].clone()})
        t = d[name][0] if name == "a" else d[name]
        t[r, slice(None) if c is None else c] = val
        v = to_dev(d)
        ref = ref_grad(d, h, base=d["x"] if name != "x" else None)
        for dt in (F32, BF):
            dx, da, db = B.lora_grad(v["x"], v["a"], v["b"], v["ids"], v["dy"],
                                     h=h.float().to(DEV), scale=v["scale"],
                                     dx_base=v["x"] if name != "x" else None, grad_dtype=dt)
            for got, want, what in ((dx, ref[0], "dx"), (da, ref[1], "da"), (db, ref[2], "db")):
                assert same(got, want), (name, what, dt)
