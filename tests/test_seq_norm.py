"""Norms around a block on the GPU against their 64-bit form."""
import pytest
import torch

import _seq_ref as R
import linear_spatial_propagation_gspn_b200 as g

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAMES = ("dy", "dr_in", "dgate", "dw_post", "db_post", "dscale", "dw_pre", "db_pre")


def make(rows, C, dtype, res, seed=0, std=1.0):
    r = torch.Generator().manual_seed(seed + rows + 3 * C)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    t = dict(y=n(rows, C) * std, gate=n(rows, C), do=n(rows, C))
    t = {k: v.to(DT[dtype]).cuda() for k, v in t.items()}
    t.update(r=n(rows, C).to(DT[res]).cuda(), dr=n(rows, C).to(DT[res]).cuda())
    t.update({k: (1 + 0.3 * n(C)).cuda() for k in ("w_post", "scale", "w_pre")}, b_post=n(C).cuda(), b_pre=n(C).cuda())
    return t


PARTS = {"all": ("gate", "w_post", "b_post", "scale", "w_pre", "b_pre"), "rms": ("gate", "w_post", "scale", "w_pre"),
         "pre": ("w_pre",), "post": ("w_post",), "gate": ("gate", "scale"), "none": ()}


def rms(t):
    return t.pow(2).mean(-1, keepdim=True).sqrt()


def bound_forward(t, ref, kw):
    """fp32 errors in units of u, as multiples of each row's size. A mean of C values summed pairwise over
    the threads and serially within one (16 values at most) is off by under 32 u of the values' size,
    a square root and quotient by 4 u, gate 48 u (its exponential's argument under 16), products 4 u:
    96 u of the normalised row's size times its weight, on top of what the norm is taken of."""
    v = R.f64(t["y"]) if "gate" not in kw else R.f64(t["y"]) * R.silu(R.f64(t["gate"]))
    size = rms(v) + v.abs()
    if "w_post" in kw:
        size = (size / rms(v) * R.f64(t["w_post"]).abs()) + (R.f64(t["b_post"]).abs() if "b_post" in kw else 0)
    if "scale" in kw:
        size = size * R.f64(t["scale"]).abs()
    return 96 * (size + ref["r_out"].abs())


SHAPES = [(1, 1), (3, 7), (5, 64), (9, 96), (4, 192), (6, 257), (2, 512), (3, 1000), (2, 1153), (3, 2048), (2, 4096), (2, 5000), (1, 8192), (2, 16384)]


@pytest.mark.parametrize("rows,C", SHAPES)
@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("parts", list(PARTS))
@pytest.mark.parametrize("center", [False, True])
def test_forward(rows, C, types, parts, center):
    if center and C == 1:
        pytest.skip("a centred row of one value is zero: its spread is eps alone")
    t = make(rows, C, *types)
    kw = {k: t[k] for k in PARTS[parts]}
    ref = R.norm(t["y"], t["r"], *(kw.get(k) for k in ("gate", "w_post", "b_post", "scale", "w_pre", "b_pre")), 1e-5, center)
    r_out, o = g.norm_forward(t["y"], t["r"], center=center, **kw)
    b = bound_forward(t, ref, kw)
    spread = 1.0
    if center:   # a row's values stand off its mean by less than their size: differences carry the size's error
        v = R.f64(t["y"]) if "gate" not in kw else R.f64(t["y"]) * R.silu(R.f64(t["gate"]))
        spread = (rms(v) / rms(v - v.mean(-1, keepdim=True))).max().item()
    R.check(r_out, ref["r_out"], b, spread, "r_out")
    assert (o is None) == ("w_pre" not in kw)
    if o is not None:
        c = ref["r_out"] - ref["r_out"].mean(-1, keepdim=True) if center else ref["r_out"]
        # the error of r_out over the row's spread, and the norm's own 96 u
        own = (b * spread).max(-1, keepdim=True).values / rms(c) + 96 * (1 + (c / rms(c)).abs()) * rms(ref["r_out"]) / rms(c)
        # a common relative error of the spread moves each value by its own size too
        own = own * (1 + (c / rms(c)).abs())
        R.check(o, ref["o"], own * R.f64(t["w_pre"]).abs() + ref["o"].abs(), 2.0, "o")


@pytest.mark.parametrize("rows,C", SHAPES + [(700, 96), (300, 1153)])
@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("parts", ["all", "rms", "pre", "gate"])
def test_backward(rows, C, types, parts):
    center = parts == "all"
    if center and (C == 1 or C > 8192):
        pytest.skip("no spread in one value; five column sums of such a row do not fit (refused)")
    t = make(rows, C, *types, seed=1)
    kw = {k: t[k] for k in PARTS[parts]}
    do = t["do"] if "w_pre" in kw else None
    got = g.norm_backward(t["y"], t["r"], t["dr"], do, center=center, **kw)
    again = g.norm_backward(t["y"], t["r"], t["dr"], do, center=center, **kw)
    ref = R.norm(t["y"], None, *(kw.get(k) for k in ("gate", "w_post", "b_post", "scale", "w_pre", "b_pre")), 1e-5, center,
                 t["r"], t["dr"], do)
    # Every element is a few sums and quotients of its row, as in the forward bound: 96 u for each norm that it
    # goes through and for the gate, of the row's largest gradient times how far values reach over their size.
    for name, a, b in zip(NAMES, got, again):
        src = {"dgate": "gate", "dw_post": "w_post", "db_post": "b_post", "dscale": "scale", "dw_pre": "w_pre", "db_pre": "b_pre"}.get(name)
        if src and src not in kw:
            assert a is None
            continue
        assert torch.equal(a, b), f"{name}: two runs differ"
        r = ref[name]
        if r.dim() == 2:
            mag = r.abs() + r.abs().max(-1, keepdim=True).values
            R.check(a, r, mag, 8 * 96.0 * reach(t, kw, center), name)
        else:
            R.check(a, r, ref[name + "_m"] + ref[name + "_m"].max(), 8 * 96.0 * reach(t, kw, center) + rows, name)


def reach(t, kw, center):
    """How much the smallest spread of a row raises errors: a row whose spread is small against its values
    turns the values' rounding into that much more of the quotient."""
    v = R.f64(t["y"]) if "gate" not in kw else R.f64(t["y"]) * R.silu(R.f64(t["gate"]))
    k = 1.0
    for w, q in (("w_post", v), ("w_pre", R.f64(t["r"]))):
        if w in kw:
            c = q - q.mean(-1, keepdim=True) if center else q
            k *= 1 + (q.abs().max(-1, keepdim=True).values / rms(c)).max().item()
    return k


def test_zero_rows_and_no_rows():
    """A row of zeros has only eps for its spread; no rows leave zero sums."""
    y = torch.zeros(2, 96, device="cuda")
    w = torch.ones(96, device="cuda")
    r_out, o = g.norm_forward(y, None, w_post=w, w_pre=w)
    assert (r_out == 0).all() and (o == 0).all()
    got = g.norm_backward(y, r_out, None, torch.ones_like(y), w_post=w, w_pre=w)
    assert all(torch.isfinite(v).all() for v in got if v is not None)
    e = torch.zeros(0, 96, device="cuda")
    r_out, o = g.norm_forward(e, e, w_pre=w)
    assert r_out.shape == o.shape == (0, 96)
    got = g.norm_backward(e, e, e, e, w_pre=w)
    assert (got[6] == 0).all()


def test_leading_axes_and_slices():
    """Rows inside wider ones, 16-byte aligned (a threads' order of its own for the sums) or not: within
    the forward bound of the 64-bit form, as test_forward derives it."""
    t = make(6, 96, "bf16", "f32")
    kw = {k: t[k] for k in ("gate", "w_post", "scale")}
    ref = R.norm(t["y"], t["r"], t["gate"], t["w_post"], None, t["scale"], None, None, 1e-5, False)
    b = bound_forward(t, ref, kw)
    for width, at in ((304, 0), (304, 8), (300, 0), (300, 1)):
        wide = torch.full((2, 3, width), float("nan"), device="cuda").bfloat16()
        y, z = wide[..., at:at + 96], wide[..., at + 104:at + 200]
        y.copy_(t["y"].view(2, 3, 96))
        z.copy_(t["gate"].view(2, 3, 96))
        r_out, _ = g.norm_forward(y, t["r"].view(2, 3, 96), **{**kw, "gate": z})
        R.check(r_out.view(6, 96), ref["r_out"], b, 1.0, f"rows of {width} from {at}")


@pytest.mark.parametrize("C", [96, 257, 1153, 2048, 4096, 5000])
@pytest.mark.parametrize("types", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_stream_in_place(C, types):
    t = make(700, C, *types, seed=5)
    kw = {k: t[k] for k in PARTS["all"]}
    want = g.norm_forward(t["y"], t["r"], center=True, **kw)
    r = t["r"].clone()
    got = g.norm_forward(t["y"], r, center=True, r_out=r, **kw)
    assert got[0] is r or got[0].data_ptr() == r.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_one_bad_row_stays_alone():
    t = make(9, 192, "f32", "f32")
    kw = {k: t[k] for k in PARTS["all"]}
    a = g.norm_forward(t["y"], t["r"], center=True, **kw)
    for bad in (float("inf"), float("nan")):
        y = t["y"].clone()
        y[4, 7] = bad
        b = g.norm_forward(y, t["r"], center=True, **kw)
        keep = torch.arange(9, device="cuda") != 4
        assert all(torch.equal(p[keep], q[keep]) for p, q in zip(a, b)) and not torch.isfinite(b[1][4]).any()


@pytest.mark.parametrize("parts", ["all", "pre", "gate"])
@pytest.mark.parametrize("use", ["both", "r_out", "o"])
def test_autograd(parts, use):
    if use == "o" and parts == "gate":
        pytest.skip("no norm before the next block: there is no o")
    t = make(5, 96, "f32", "f32", seed=2)
    kw = {k: t[k].clone().requires_grad_(True) for k in PARTS[parts]}
    y, r = (t[k].clone().requires_grad_(True) for k in ("y", "r"))
    r_out, o = g.block_norm(y, r, center=True, **kw)
    dr = t["dr"] if use != "o" else None
    do = t["do"] if use != "r_out" and o is not None else None
    torch.autograd.backward(*zip(*[(a, b) for a, b in ((r_out, dr), (o, do)) if b is not None]))
    zero = torch.zeros_like(t["do"])
    ref = R.norm(t["y"], None, *(kw.get(k) for k in ("gate", "w_post", "b_post", "scale", "w_pre", "b_pre")), 1e-5, True, r_out,
                 zero if dr is None else dr, None if o is None else zero if do is None else do)
    src = dict(dy=y, dr_in=r, dgate=kw.get("gate"), dw_post=kw.get("w_post"), db_post=kw.get("b_post"), dscale=kw.get("scale"),
               dw_pre=kw.get("w_pre"), db_pre=kw.get("b_pre"))
    for name, leaf in src.items():
        if leaf is not None:
            R.check(leaf.grad, ref[name], ref[name].abs() + ref[name].abs().max() + 1, 8 * 96 * reach(t, kw, True), name)
