"""Causal convolution on the GPU against its 64-bit form: prompts, gradients, single tokens."""
import pytest
import torch

import _seq_ref as R
import linear_spatial_propagation_gspn_b200 as g

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# u: a bias and K <= 4 products added one by one, 6 roundings; silu and its slope: exponential (2 u and its
# argument's rounding, |v| u <= 30 u here), quotient 2 u, products 4 u
F = 48


def make(B, L, C, K, dtype, seqs=None, bias=True, state=True, seed=0):
    r = torch.Generator().manual_seed(seed + 17 * L + C + K)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    S = B if seqs is None else seqs
    t = dict(x=n(B, L, C), dy=n(B, L, C), state0=n(S, K - 1, C) if state else None, dstate=n(S, K - 1, C))
    t = {k: v if v is None else v.to(DT[dtype]).cuda() for k, v in t.items()}
    t.update(w=n(C, K).cuda(), bias=n(C).cuda() if bias else None)
    return t


SHAPES = [(1, 1, 1, 2), (2, 3, 5, 4), (1, 17, 8, 3), (3, 33, 40, 4), (2, 70, 136, 4), (1, 129, 33, 2), (1, 40, 512, 4)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("full", [True, False])
def test_prompt_and_gradients(shape, dtype, full):
    t = make(*shape, dtype, bias=full, state=full)
    ds = t["dstate"] if full else None
    ref = R.conv(t["x"], t["w"], t["bias"], full, None, t["state0"], t["dy"], ds)
    state = torch.empty_like(t["dstate"])
    y = g.conv_forward(t["x"], t["w"], t["bias"], silu=full, state0=t["state0"], state=state)
    R.check(y, ref["y"], ref["y_m"], F, "y")
    assert torch.equal(R.f64(state), ref["state"])
    got = g.conv_backward(t["x"], t["w"], t["bias"], t["dy"], silu=full, state0=t["state0"], dstate=ds)
    again = g.conv_backward(t["x"], t["w"], t["bias"], t["dy"], silu=full, state0=t["state0"], dstate=ds)
    for name, a, b in zip(("dx", "dw", "db", "ds"), got, again):
        if a is None:
            assert not full and name in ("db", "ds")
            continue
        assert torch.equal(a, b), f"{name}: two runs differ"
        R.check(a, ref[name], ref[name + "_m"], F + shape[0] * shape[1], name)


@pytest.mark.parametrize("cu,L", [([0, 7, 7, 40, 41, 43], 43), ([3, 20, 20, 36], 45), ([0, 0, 0], 9), ([0, 31, 33, 34, 96], 96),
                                  ([0, 1, 2, 3, 4, 5, 6], 70)])
@pytest.mark.parametrize("K", [2, 4])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("state", [True, False])
def test_packed(cu, L, K, dtype, state):
    t = make(1, L, 40, K, dtype, seqs=len(cu) - 1, state=state, seed=1)
    a, b = cu[0], cu[-1]
    for k in ("x", "dy"):
        t[k][:, :a] = float("nan")
        t[k][:, b:] = float("nan")
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ref = R.conv(t["x"], t["w"], t["bias"], True, cu, t["state0"], t["dy"], t["dstate"])
    y, last = torch.full_like(t["x"], 7.0), torch.empty_like(t["dstate"])
    g.conv_forward(t["x"], t["w"], t["bias"], cu=c, state0=t["state0"], y=y, state=last)
    out = (torch.full_like(y, 7.0), torch.empty_like(t["w"]), torch.empty_like(t["bias"]), torch.empty_like(last) if state else None)
    g.conv_backward(t["x"], t["w"], t["bias"], t["dy"], cu=c, state0=t["state0"], dstate=t["dstate"], out=out)
    inside = torch.zeros(1, L, dtype=torch.bool)
    inside[:, a:b] = True
    assert torch.equal(R.f64(last), ref["state"])
    for name, v in (("y", y), ("dx", out[0])):
        assert (v.cpu()[~inside] == 7).all(), f"{name}: tokens outside were written"
        R.check(v.cpu()[inside], ref[name][inside], ref[name + "_m"][inside], F, name)
    for name, v in zip(("dw", "db", "ds"), out[1:]):
        if v is not None:
            R.check(v, ref[name], ref[name + "_m"], F + L, name)


def test_no_tokens():
    t = make(2, 0, 8, 4, "f32")
    y = g.conv_forward(t["x"], t["w"], t["bias"], state0=t["state0"], state=t["dstate"])
    assert y.shape == (2, 0, 8) and torch.equal(t["dstate"], t["state0"])
    _, dw, db, ds = g.conv_backward(t["x"], t["w"], t["bias"], t["dy"], state0=t["state0"], dstate=t["dstate"])
    assert (dw == 0).all() and (db == 0).all() and torch.equal(ds, t["dstate"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_slices_and_state_in_place(dtype, pad):
    """x as a slice of wider rows; a prompt in pieces, the state in one buffer; then single tokens."""
    B, L, C = 2, 50, 48
    t = make(B, L, C, 4, dtype, seed=2)
    wide = torch.full((B, L + 2, C + 8 + pad), float("nan"), dtype=DT[dtype], device="cuda")
    x = wide[:, 1:L + 1, pad:pad + C]
    x.copy_(t["x"])
    whole = g.conv_forward(t["x"], t["w"], t["bias"], state0=t["state0"])
    state = t["state0"].clone()
    ys = [g.conv_forward(x[:, a:b], t["w"], t["bias"], state0=state, state=state) for a, b in ((0, 2), (2, 30), (30, 47))]
    ys += [g.conv_step(x[:, i], t["w"], t["bias"], state)[:, None] for i in range(47, 50)]
    assert torch.equal(torch.cat(ys, 1), whole)
    assert torch.equal(state, t["x"][:, -3:])


@pytest.mark.parametrize("shape", [(1, 1, 2), (3, 33, 3), (130, 64, 4), (2, 2048, 4)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", [True, False])
def test_step(shape, dtype, act):
    B, C, K = shape
    t = make(B, 1, C, K, dtype, bias=act, seed=3)
    ref = R.conv(t["x"], t["w"], t["bias"], act, None, t["state0"])
    slots = B + 2
    pool = torch.randn(slots, K - 1, C, device="cuda").to(DT[dtype])
    idx = torch.randperm(slots, generator=torch.Generator().manual_seed(B))[:B].to(torch.int32).cuda()
    pool[idx.long()] = t["state0"]
    before = pool.clone()
    y = g.conv_step(t["x"][:, 0], t["w"], t["bias"], pool, idx=idx, silu=act)
    R.check(y, ref["y"][:, 0], ref["y_m"][:, 0], F, "y")
    assert torch.equal(R.f64(pool[idx.long()]), ref["state"])
    rest = torch.ones(slots, dtype=torch.bool, device="cuda")
    rest[idx.long()] = False
    assert torch.equal(pool[rest], before[rest])


def test_step_repeated_and_missing_slots():
    C, idx = 40, [2, 0, 2, -1, 2, 9]
    t = make(1, len(idx), C, 4, "bf16", seed=4)
    pool = torch.randn(4, 3, C, device="cuda").bfloat16()
    before = pool.clone()
    y = torch.full((len(idx), C), 7.0, device="cuda").bfloat16()
    g.conv_step(t["x"][0], t["w"], t["bias"], pool, idx=torch.tensor(idx, dtype=torch.int32, device="cuda"), y=y)
    for slot in (0, 2):
        rows = [i for i, v in enumerate(idx) if v == slot]
        ref = R.conv(t["x"][:, rows], t["w"], t["bias"], True, None, before[slot][None])
        R.check(y[rows], ref["y"][0], ref["y_m"][0], F, "y")
        assert torch.equal(R.f64(pool[slot]), ref["state"][0])
    assert (y[[3, 5]] == 7).all() and torch.equal(pool[[1, 3]], before[[1, 3]])


def test_far_values():
    x = torch.tensor([-3e38, -200.0, -90.0, -0.0, 0.0, 90.0, 200.0, 3e38], device="cuda").reshape(1, 8, 1).contiguous()
    w = torch.tensor([[0.0, 1.0]], device="cuda")
    y = g.conv_forward(x, w)
    ref = R.silu(R.f64(x))
    assert torch.allclose(R.f64(y), ref, rtol=1e-6, atol=1e-30)


@pytest.mark.parametrize("cu", [None, [0, 9, 30]])
def test_autograd(cu):
    B = 2 if cu is None else 1
    t = make(B, 33, 40, 4, "f32", seqs=None if cu is None else 2, seed=5)
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    ref = R.conv(t["x"], t["w"], t["bias"], True, cu, t["state0"], t["dy"], t["dstate"])
    leaf = [t[k].clone().requires_grad_(True) for k in ("x", "w", "bias", "state0")]
    y, state = g.causal_conv(*leaf[:3], cu=c, state0=leaf[3], return_state=True)
    torch.autograd.backward([y, state], [t["dy"], t["dstate"]])
    for name, v in zip(("dx", "dw", "db", "ds"), leaf):
        R.check(v.grad, ref[name], ref[name + "_m"], F + 33 * B, name)
    if cu is not None:
        assert (y[:, cu[-1]:] == 0).all() and (leaf[0].grad[:, cu[-1]:] == 0).all()
    g.causal_conv(leaf[0].detach(), leaf[1].detach().requires_grad_(True)).sum().backward()
