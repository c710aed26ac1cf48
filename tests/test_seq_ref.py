"""The 64-bit forms that the token-sequence kernels are held to: gradients by formula against central
differences, packed sequences against each one alone."""
import pytest
import torch

import _seq_ref as R

H = 1e-5


def differences(f, leaves, weights):
    """d sum(weights . f) / d leaf by central differences, for every leaf element."""
    def total():
        return sum((w * v).sum() for w, v in zip(weights, f()) if w is not None)
    out = []
    for t in leaves:
        g, flat = torch.zeros_like(t), t.view(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + H
            up = total()
            flat[i] = keep - H
            g.view(-1)[i] = (up - total()) / (2 * H)
            flat[i] = keep
        out.append(g)
    return out


def near(a, b, what):
    # central differences of O(1) functions: H^2 truncation and 2^-53 / H cancellation, some 1e-9 together
    assert (a - b).abs().max() <= 1e-7 * max(1.0, b.abs().max()), what


def rand(g, *s):
    return torch.randn(*s, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("cu", [None, [0, 2, 2, 5], [1, 4]])
@pytest.mark.parametrize("act", [True, False])
def test_conv_gradients(cu, act):
    g = torch.Generator().manual_seed(3)
    B, L, C, K = (2 if cu is None else 1), 5, 3, 4
    S = B if cu is None else len(cu) - 1
    x, w, b, s0 = rand(g, B, L, C), rand(g, C, K), rand(g, C), rand(g, S, K - 1, C)
    dy, ds = rand(g, B, L, C), rand(g, S, K - 1, C)
    ref = R.conv(x, w, b, act, cu, s0, dy, ds)
    f = lambda: (lambda o: (o["y"], o["state"]))(R.conv(x, w, b, act, cu, s0))  # noqa: E731
    for name, got in zip(("dx", "dw", "db", "ds"), differences(f, (x, w, b, s0), (dy, ds))):
        near(got, ref[name], name)


@pytest.mark.parametrize("cu", [None, [0, 2, 2, 5]])
@pytest.mark.parametrize("gate,soft", [(True, True), (False, False)])
def test_scan_gradients(cu, gate, soft):
    g = torch.Generator().manual_seed(4)
    B, L, C, G, N = (2 if cu is None else 1), 5, 4, 2, 3
    S = B if cu is None else len(cu) - 1
    x, dt, A, Bm, Cm = rand(g, B, L, C), rand(g, B, L, C), -rand(g, C, N).abs(), rand(g, B, L, G, N), rand(g, B, L, G, N)
    D, z, bias, h0 = rand(g, C), rand(g, B, L, C) if gate else None, rand(g, C), rand(g, S, C, N)
    if not soft:
        dt.abs_()
    dy, dh = rand(g, B, L, C), rand(g, S, C, N)
    ref = R.scan(x, dt, A, Bm, Cm, D, z, bias, soft, cu, h0, dy, dh)
    f = lambda: (lambda o: (o["y"], o["h"]))(R.scan(x, dt, A, Bm, Cm, D, z, bias, soft, cu, h0))  # noqa: E731
    leaves = dict(dx=x, ddt=dt, dA=A, dB=Bm, dC=Cm, dD=D, dbias=bias, dh0=h0)
    if gate:
        leaves["dz"] = z
    for name, got in zip(leaves, differences(f, list(leaves.values()), (dy, dh))):
        near(got, ref[name], name)


@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_norm_gradients(center, gate):
    g = torch.Generator().manual_seed(5)
    n, C = 3, 6
    y, r, z = rand(g, n, C), rand(g, n, C), rand(g, n, C) if gate else None
    w1, b1, s, w2, b2, dr, do = rand(g, C), rand(g, C), rand(g, C), rand(g, C), rand(g, C), rand(g, n, C), rand(g, n, C)
    full = R.norm(y, r, z, w1, b1, s, w2, b2, 1e-3, center)
    ref = R.norm(y, r, z, w1, b1, s, w2, b2, 1e-3, center, full["r_out"], dr, do)
    f = lambda: (lambda o: (o["r_out"], o["o"]))(R.norm(y, r, z, w1, b1, s, w2, b2, 1e-3, center))  # noqa: E731
    leaves = dict(dy=y, dr_in=r, dw_post=w1, db_post=b1, dscale=s, dw_pre=w2, db_pre=b2)
    if gate:
        leaves["dgate"] = z
    for name, got in zip(leaves, differences(f, list(leaves.values()), (dr, do))):
        near(got, ref[name], name)


def test_packed_is_each_alone():
    g = torch.Generator().manual_seed(6)
    C, N, cu = 4, 2, [0, 3, 3, 7]
    x, dt, A = rand(g, 1, 7, C), rand(g, 1, 7, C), -rand(g, C, N).abs()
    Bm, Cm = rand(g, 1, 7, 1, N), rand(g, 1, 7, 1, N)
    packed = R.scan(x, dt, A, Bm, Cm, None, None, None, True, cu, None)
    for q, (a, b) in enumerate(zip(cu, cu[1:])):
        if b > a:
            one = R.scan(x[:, a:b], dt[:, a:b], A, Bm[:, a:b], Cm[:, a:b], None, None, None, True, None, None)
            assert torch.equal(one["y"], packed["y"][:, a:b]) and torch.equal(one["h"][0], packed["h"][q])
