"""Token-sequence operators where offsets pass 32 bits: tokens, rows and slots more than 2^31 elements from
their tensor's start give the bits that they give by themselves."""
import pytest
import torch

import _seq_ref as R
import linear_spatial_propagation_gspn_b200 as g

pytestmark = pytest.mark.gpu
L, C, N, G = 1_050_000, 2048, 4, 1                                # L C > 2^31
FROM = L - 75
CU = [0, 30, 30, 70]                                              # within the last tokens; five behind the last sequence


@pytest.fixture(scope="module")
def data():
    assert L * C > 2 ** 31
    gen = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    t = dict(x=torch.empty(1, L, C, dtype=torch.bfloat16, device="cuda"), bc=torch.empty(1, L, G, N, dtype=torch.bfloat16, device="cuda"))
    for v in t.values():
        v[:, FROM:] = n(1, L - FROM, *v.shape[2:]).bfloat16()
    t.update(w=n(C, 4), A=-n(C, N).abs(), D=n(C), bias=n(C) - 3, w_post=n(C), w_pre=n(C), h0=n(3, C, N), state0=n(3, 3, C).bfloat16())
    for at, name in ((FROM, "far"), (0, "near")):
        t[name] = torch.tensor([at + v for v in CU], dtype=torch.int32, device="cuda")
    yield t
    t.clear()
    torch.cuda.empty_cache()


def same(far, near):
    for i, (a, b) in enumerate(zip(far, near)):
        if b is None:
            assert a is None
        elif b.dim() >= 3 and b.shape[1] == L - FROM:             # tokens: those of the sequences
            assert torch.equal(a[:, FROM:FROM + CU[-1]], b[:, :CU[-1]]), i
        else:
            assert torch.equal(a, b), i


def test_convolution(data):
    t, x = data, data["x"]
    near = x[:, FROM:].clone()
    got, want = [], []
    for v, cu, out in ((x, t["far"], got), (near, t["near"], want)):
        y, state = torch.empty_like(v), torch.empty_like(t["state0"])
        out.append(g.conv_forward(v, t["w"], t["bias"], cu=cu, state0=t["state0"], y=y, state=state))
        out.append(state)
        dx, dw, db, ds = g.conv_backward(v, t["w"], t["bias"], y, cu=cu, state0=t["state0"], dstate=state)
        out.extend((dx, ds))
    same(got, want)
    # how many tokens are summed at a time depends on how many there are: the filter's gradients by their bound
    ref = R.conv(near, t["w"], t["bias"], True, CU, t["state0"], want[0], want[1])
    R.check(dw, ref["dw"], ref["dw_m"], 48 + CU[-1], "near dw")
    dw, db = g.conv_backward(x, t["w"], t["bias"], got[0], cu=t["far"], state0=t["state0"], dstate=got[1])[1:3]
    R.check(dw, ref["dw"], ref["dw_m"], 48 + CU[-1], "dw")
    R.check(db, ref["db"], ref["db_m"], 48 + CU[-1], "db")


def test_scan(data):
    """Into how many pieces sequences are cut depends on how many tokens there are, so here the 64-bit form tells
    what is right, with the bounds of the operator's own tests."""
    t = data
    x, bc, at = t["x"], t["bc"], slice(FROM, FROM + CU[-1])
    kw = dict(D=t["D"], z=x, dt_bias=t["bias"], cu=t["far"], h0=t["h0"])
    h = torch.empty_like(t["h0"])
    y, save = g.ssm_forward_save(x, x, t["A"], bc, bc, h=h, **kw)
    got = g.ssm_backward(x, x, t["A"], bc, bc, y, save, dh=h, **kw)
    near, nbc, dy = x[:, at].clone(), bc[:, at].clone(), y[:, at].clone()
    ref = R.scan(near, near, t["A"], nbc, nbc, t["D"], near, t["bias"], True, CU, t["h0"], dy, h)
    f = R.scan_factor(40, N, C)
    R.check(y[:, at], ref["y"], ref["y_m"], f, "y")
    R.check(h, ref["h"], ref["h_m"], f, "h")
    for name, v in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0"), got):
        v = v[:, at] if v.dim() >= 3 and v.shape[1] == L else v
        R.check(v, ref[name], ref[name + "_m"], f + CU[-1], name)


def test_norms(data):
    t, x = data, data["x"][0]
    near = x[FROM:].clone()
    kw = dict(gate=None, w_post=t["w_post"], w_pre=t["w_pre"])
    x[:FROM] = 0
    far, by_itself = g.norm_forward(x, x, **kw), g.norm_forward(near, near, **kw)
    for a, b in zip(far, by_itself):
        assert torch.equal(a[FROM:], b)
    del a, far
    got, want = g.norm_backward(x, x, x, x, **kw), g.norm_backward(near, near, near, near, **kw)
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a[FROM:], b)


def test_slots():
    """The last of more slots than 2^31 elements hold."""
    C, N, rows = 8192, 64, 3
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    x, bc, A, D, w = n(rows, C), n(rows, 1, N), -n(C, N).abs(), n(C), n(C, 4)
    slots = 2 ** 31 // (C * N) + 2
    pool, few, at = torch.empty(slots, C, N, device="cuda"), n(rows, C, N), torch.tensor([slots - 1, 0, slots - 2], dtype=torch.int32).cuda()
    pool[at.long()] = few
    a = g.ssm_step(x, x, A, bc, bc, pool, D=D, idx=at)
    b = g.ssm_step(x, x, A, bc, bc, few, D=D)
    assert torch.equal(a, b) and torch.equal(pool[at.long()], few)
    del pool
    slots = 2 ** 31 // (3 * C) + 2
    pool, few, at = torch.empty(slots, 3, C, dtype=torch.bfloat16, device="cuda"), n(rows, 3, C).bfloat16(), \
        torch.tensor([slots - 1, 0, slots - 2], dtype=torch.int32).cuda()
    pool[at.long()] = few
    x = x.bfloat16()
    a, b = g.conv_step(x, w, None, pool, idx=at), g.conv_step(x, w, None, few)
    assert torch.equal(a, b) and torch.equal(pool[at.long()], few)
    del pool
    torch.cuda.empty_cache()
