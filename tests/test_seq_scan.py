"""Selective scan on the GPU against its 64-bit form: prompts, gradients, single tokens; every state
width class, odd sizes, groups, packed sequences, pieces of long sequences."""
import pytest
import torch

import _seq_ref as R
import linear_spatial_propagation_gspn_b200 as g

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0")


def make(B, L, C, G, N, dtype, seqs=None, gate=True, D=True, bias=True, h0=True, seed=0):
    r = torch.Generator().manual_seed(seed + 131 * L + 7 * C + N)
    n = lambda *s, k=1.0: torch.randn(*s, generator=r) * k  # noqa: E731
    S = B if seqs is None else seqs
    t = dict(x=n(B, L, C), dt=n(B, L, C, k=0.5), Bm=n(B, L, G, N), Cm=n(B, L, G, N), z=n(B, L, C) if gate else None, dy=n(B, L, C))
    t = {k: v if v is None else v.to(DT[dtype]).cuda() for k, v in t.items()}
    f = dict(A=-torch.rand(C, N, generator=r) * 4 - 0.05, D=n(C) if D else None, dt_bias=n(C) * 0.5 - 1 if bias else None,
             h0=n(S, C, N) if h0 else None, dh=n(S, C, N))
    t.update({k: v if v is None else v.cuda() for k, v in f.items()})
    return t


def args(t):
    return (t["x"], t["dt"], t["A"], t["Bm"], t["Cm"])


def opts(t, **kw):
    return dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], h0=t["h0"], **kw)


def reference(t, soft=True, cu=None, grads=False):
    return R.scan(*args(t), t["D"], t["z"], t["dt_bias"], soft, cu, t["h0"], t["dy"] if grads else None, t["dh"] if grads else None)


def factor(t, cu=None):
    B, L, C = t["x"].shape
    return R.scan_factor(max([1] + [b - a for _, a, b in R.spans(B, L, cu)]), t["A"].shape[1], C)


SHAPES = [(1, 1, 1, 1, 1), (1, 5, 33, 1, 5), (2, 37, 40, 2, 16), (3, 33, 32, 1, 8), (1, 64, 64, 1, 16), (2, 70, 72, 2, 24),
          (1, 35, 36, 1, 64), (1, 18, 10, 5, 33), (1, 400, 40, 1, 16), (1, 333, 24, 2, 12)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("full", [True, False])
def test_prompt(shape, dtype, full):
    t = make(*shape, dtype, gate=full, D=full, bias=full, h0=full)
    if not full:
        t["dt"].abs_()
    h = torch.full((shape[0], shape[2], shape[4]), float("nan"), device="cuda")
    y = g.ssm_forward(*args(t), **opts(t, softplus=full, h=h))
    y2, hsave = g.ssm_forward_save(*args(t), **opts(t, softplus=full))
    ref = reference(t, full)
    R.check(y, ref["y"], ref["y_m"], factor(t), "y")
    R.check(h, ref["h"], ref["h_m"], factor(t), "h")
    assert torch.equal(y, y2), "keeping the states changed y"


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("full", [True, False])
def test_gradients(shape, dtype, full):
    t = make(*shape, dtype, gate=full, D=full, bias=full, h0=full, seed=1)
    if not full:
        t["dt"].abs_()
        t["dh"] = None
    _, hsave = g.ssm_forward_save(*args(t), **opts(t, softplus=full))
    kw = opts(t, softplus=full, dh=t["dh"])
    got = g.ssm_backward(*args(t), t["dy"], hsave, **kw)
    again = g.ssm_backward(*args(t), t["dy"], hsave, **kw)
    ref = reference(t, full, grads=True)
    for name, a, b in zip(GRADS, got, again):
        if a is None:
            assert not full and name in ("dD", "dz", "dbias", "dh0")
            continue
        assert torch.equal(a, b), f"{name}: two runs differ"
        R.check(a, ref[name], ref[name + "_m"], factor(t) + shape[0] * shape[1], name)


@pytest.mark.parametrize("cu,L", [([0, 7, 7, 40, 41], 41), ([3, 20, 20, 36], 45), ([0, 0, 0], 9), ([0, 300, 301, 640], 640), ([0, 500], 520)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed(cu, L, dtype):
    """Sequences of no, one and many tokens; tokens in none stay out of everything, whatever they hold."""
    t = make(1, L, 40, 2, 16, dtype, seqs=len(cu) - 1, seed=2)
    a, b = cu[0], cu[-1]
    for k in ("x", "dt", "Bm", "Cm", "z", "dy"):
        t[k][:, :a] = float("nan")
        t[k][:, b:] = float("nan")
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ref = reference(t, cu=cu, grads=True)
    y = torch.full_like(t["x"], 7.0)
    h = torch.empty_like(t["h0"])
    _, hsave = g.ssm_forward_save(*args(t), **opts(t, cu=c, y=y, h=h))
    out = [None if v is None else torch.full_like(v, 7.0) for v in
           (t["x"], t["dt"], t["A"], t["Bm"], t["Cm"], t["D"], t["z"], t["dt_bias"], t["h0"])]
    got = g.ssm_backward(*args(t), t["dy"], hsave, **opts(t, cu=c, dh=t["dh"], out=out))
    f = factor(t, cu) + L
    inside = torch.zeros(1, L, dtype=torch.bool)
    inside[:, a:b] = True
    R.check(y.cpu()[inside], ref["y"][inside], ref["y_m"][inside], f, "y")
    R.check(h, ref["h"], ref["h_m"], f, "h")
    assert (y.cpu()[~inside] == 7).all(), "tokens outside were written"
    for name, v in zip(GRADS, got):
        r, m = ref[name], ref[name + "_m"]
        if name in ("dx", "ddt", "dB", "dC", "dz"):
            assert (v.cpu()[~inside] == 7).all(), f"{name}: tokens outside were written"
            v, r, m = v.cpu()[inside], r[inside], m[inside]
        R.check(v, r, m, f, name)


def test_no_tokens():
    t = make(2, 0, 8, 1, 4, "f32")
    h = torch.empty_like(t["h0"])
    y, hsave = g.ssm_forward_save(*args(t), **opts(t, h=h))
    assert y.shape == (2, 0, 8) and torch.equal(h, t["h0"])
    got = dict(zip(GRADS, g.ssm_backward(*args(t), t["dy"], hsave, **opts(t, dh=t["dh"]))))
    assert torch.equal(got["dh0"], t["dh"])
    for name in ("dA", "dD", "dbias"):
        assert (got[name] == 0).all()


@pytest.mark.parametrize("L", [37, 400])
def test_state_in_place_and_pieces_of_a_prompt(L):
    """A prompt read in two calls, the state going on in its own buffer, is the prompt read in one."""
    t = make(1, L, 40, 1, 16, "f32", seed=3)
    ref = reference(t)
    h, cut = t["h0"].clone(), L // 3
    ys = []
    for a, b in ((0, cut), (cut, L)):
        part = {k: t[k][:, a:b] for k in ("x", "dt", "Bm", "Cm", "z")}
        ys.append(g.ssm_forward(part["x"], part["dt"], t["A"], part["Bm"], part["Cm"], D=t["D"], z=part["z"], dt_bias=t["dt_bias"],
                                h0=h, h=h))
    R.check(torch.cat(ys, 1), ref["y"], ref["y_m"], factor(t), "y")
    R.check(h, ref["h"], ref["h_m"], factor(t), "h")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_slices_of_a_projection(dtype, pad):
    """Inputs that lie side by side in wider rows, 16-byte aligned or not."""
    B, L, C, N = 2, 50, 48, 16
    t = make(B, L, C, 1, N, dtype, seed=4)
    wide = torch.full((B, L + 2, 3 * C + 2 * N + pad), float("nan"), dtype=DT[dtype], device="cuda")
    at, parts = pad, {}
    for k, n in (("x", C), ("Bm", N), ("dt", C), ("Cm", N), ("z", C)):
        parts[k] = wide[:, 1:L + 1, at:at + n]
        parts[k].copy_(t[k].reshape(B, L, n))
        at += n
    for k in ("Bm", "Cm"):
        parts[k] = parts[k].unflatten(2, (1, N))
    s = {**t, **parts}
    y1, save1 = g.ssm_forward_save(*args(t), **opts(t))
    y2, save2 = g.ssm_forward_save(*args(s), **opts(s))
    assert torch.equal(y1, y2)
    for name, a, b in zip(GRADS, g.ssm_backward(*args(t), t["dy"], save1, **opts(t)), g.ssm_backward(*args(s), t["dy"], save2, **opts(s))):
        assert torch.equal(a, b), name
    part = {k: v[:, 5] for k, v in s.items() if k in ("x", "dt", "Bm", "Cm", "z")}
    hs = [t["h0"].clone() for _ in range(2)]
    ys = [g.ssm_step(p["x"], p["dt"], t["A"], p["Bm"], p["Cm"], h, D=t["D"], z=p["z"], dt_bias=t["dt_bias"])
          for p, h in ((part, hs[0]), ({k: v.contiguous() for k, v in part.items()}, hs[1]))]
    assert torch.equal(*ys) and torch.equal(*hs)


@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (3, 33, 1, 5), (5, 40, 2, 16), (4, 72, 2, 24), (2, 36, 1, 64), (130, 64, 1, 16)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("full", [True, False])
def test_step(shape, dtype, full):
    B, C, G, N = shape
    t = make(B, 1, C, G, N, dtype, gate=full, D=full, bias=full, seed=5)
    if not full:
        t["dt"].abs_()
    ref = reference(t, full)
    s = {k: t[k] if t[k] is None else t[k][:, 0] for k in ("x", "dt", "Bm", "Cm", "z")}
    slots = B + 3
    pool = torch.randn(slots, C, N, device="cuda")
    idx = torch.randperm(slots, generator=torch.Generator().manual_seed(B))[:B].to(torch.int32).cuda()
    pool[idx.long()] = t["h0"]
    before = pool.clone()
    y = g.ssm_step(s["x"], s["dt"], t["A"], s["Bm"], s["Cm"], pool, D=t["D"], z=s["z"], dt_bias=t["dt_bias"], softplus=full, idx=idx)
    R.check(y, ref["y"][:, 0], ref["y_m"][:, 0], factor(t), "y")
    R.check(pool[idx.long()], ref["h"], ref["h_m"], factor(t), "h")
    rest = torch.ones(slots, dtype=torch.bool, device="cuda")
    rest[idx.long()] = False
    assert torch.equal(pool[rest], before[rest]), "a slot that no row names was written"


def test_step_repeated_and_missing_slots():
    """A slot named three times takes its tokens in row order; rows without a slot are left alone."""
    C, N, idx = 40, 16, [2, 0, 2, -1, 2, 9]
    t = make(1, len(idx), C, 1, N, "f32", seed=6)
    s = {k: t[k][0] for k in ("x", "dt", "Bm", "Cm", "z")}
    pool = torch.randn(4, C, N, device="cuda")
    before = pool.clone()
    y = torch.full((len(idx), C), 7.0, device="cuda")
    g.ssm_step(s["x"], s["dt"], t["A"], s["Bm"], s["Cm"], pool, D=t["D"], z=s["z"], dt_bias=t["dt_bias"], y=y,
               idx=torch.tensor(idx, dtype=torch.int32, device="cuda"))
    for slot in (0, 2):
        rows = [i for i, v in enumerate(idx) if v == slot]
        one = {k: t[k][:, rows] for k in ("x", "dt", "Bm", "Cm", "z")}
        ref = R.scan(one["x"], one["dt"], t["A"], one["Bm"], one["Cm"], t["D"], one["z"], t["dt_bias"], True, None, before[slot][None])
        R.check(y[rows], ref["y"][0], ref["y_m"][0], factor(t), "y")
        R.check(pool[slot], ref["h"][0], ref["h_m"][0], factor(t), "h")
    assert (y[[3, 5]] == 7).all() and torch.equal(pool[[1, 3]], before[[1, 3]])


def test_steps_continue_a_prompt():
    t = make(2, 45, 40, 1, 16, "bf16", seed=7)
    ref = reference(t)
    h = torch.empty_like(t["h0"])
    p = {k: t[k][:, :40] for k in ("x", "dt", "Bm", "Cm", "z")}
    g.ssm_forward(p["x"], p["dt"], t["A"], p["Bm"], p["Cm"], D=t["D"], z=p["z"], dt_bias=t["dt_bias"], h0=t["h0"], h=h)
    for i in range(40, 45):
        s = {k: t[k][:, i] for k in ("x", "dt", "Bm", "Cm", "z")}
        y = g.ssm_step(s["x"], s["dt"], t["A"], s["Bm"], s["Cm"], h, D=t["D"], z=s["z"], dt_bias=t["dt_bias"])
        R.check(y, ref["y"][:, i], ref["y_m"][:, i], factor(t), f"token {i}")
    R.check(h, ref["h"], ref["h_m"], factor(t), "h")


def test_far_steps():
    """Steps from nearly nothing to so large that the state is forgotten; infinities and NaN stay in
    their channel."""
    t = make(1, 40, 64, 1, 16, "f32", seed=8)
    t["dt"] = torch.linspace(-120, 120, 40 * 64, device="cuda").reshape(1, 64, 40).transpose(1, 2).contiguous()
    t["dt_bias"] = None
    ref = reference(t)
    y = g.ssm_forward(*args(t), **opts(t))
    # |d A| goes to 480 here, where the decay is nothing; its error d(exp(-v)) = v exp(-v) u stays under u
    R.check(y, ref["y"], ref["y_m"], factor(t), "y")
    for bad in (float("inf"), float("nan")):
        x = t["x"].clone()
        x[0, 3, 5] = bad
        yb = g.ssm_forward(x, *args(t)[1:], **opts(t))
        keep = torch.arange(64, device="cuda") != 5
        assert torch.equal(yb[:, :, keep], y[:, :, keep]) and torch.equal(yb[:, :3], y[:, :3])
        assert not torch.isfinite(yb[0, 3, 5])


@pytest.mark.parametrize("cu", [None, [0, 9, 30]])
def test_autograd(cu):
    B = 2 if cu is None else 1
    t = make(B, 33, 40, 2, 16, "f32", seqs=None if cu is None else 2, seed=9)
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    ref = reference(t, cu=cu, grads=True)
    names = ("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0")
    leaf = {k: t[k].clone().requires_grad_(True) for k in names}
    y, h = g.selective_scan(leaf["x"], leaf["dt"], leaf["A"], leaf["Bm"], leaf["Cm"], leaf["D"], leaf["z"], leaf["dt_bias"], cu=c,
                            h0=leaf["h0"], return_state=True)
    if cu is not None:
        assert (y[:, cu[-1]:] == 0).all()
    torch.autograd.backward([y, h], [t["dy"], t["dh"]])
    for k, name in zip(names, GRADS):
        R.check(leaf[k].grad, ref[name], ref[name + "_m"], factor(t, cu) + 33 * B, name)
    # a broadcast gradient of the output, and no use of the state
    y = g.selective_scan(*(leaf[k].detach().requires_grad_(True) for k in names[:5]), cu=c)
    y.sum().backward()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["rates", "steps"])
def test_states_that_do_not_decay_stay_as_they_are(dtype, kind):
    """A rate or a step of zero decays by one exactly, over any number of tokens: prompt, gradient and token."""
    t = make(2, 500, 48, 1, 16, dtype, seed=11)
    t["Bm"].zero_() if kind == "rates" else t["dt"].zero_()
    A = torch.zeros_like(t["A"]) if kind == "rates" else t["A"]
    kw = dict(D=t["D"], z=t["z"], h0=t["h0"], softplus=False)
    h = torch.empty_like(t["h0"])
    dt = t["dt"].abs()
    y, save = g.ssm_forward_save(t["x"], dt, A, t["Bm"], t["Cm"], h=h, **kw)
    assert torch.equal(h, t["h0"])
    dh0 = g.ssm_backward(t["x"], dt, A, t["Bm"], t["Cm"], torch.zeros_like(y), save, dh=t["dh"], **kw)[-1]
    assert torch.equal(dh0, t["dh"])
    g.ssm_step(t["x"][:, 0], dt[:, 0], A, t["Bm"][:, 0], t["Cm"][:, 0], h, D=t["D"], z=t["z"][:, 0], softplus=False)
    assert torch.equal(h, t["h0"])
