"""The scan's errors where they add up: slow channels over thousands of tokens, and whole fp32 outputs by their norm.

u = 2^-24. A token rounds a state twice, decay and update; together that is 1.2 u rms at most (the decay's own
error is 0.5 u rms, its product and sum half a step each at most), and over T tokens of changing steps sqrt(T) 1.2 u.
What a token's decay is off by on average adds up T times: u / 32 is allowed of it. A norm over many channels and
states sees these rms values, not the worst element's.
"""
import pytest
import torch

import _seq_ref as R
import linear_spatial_propagation_gspn_b200 as g

pytestmark = pytest.mark.gpu


def steps(T):
    """The relative error of T tokens' decays and updates."""
    return (1.2 * T ** 0.5 + T / 32) * R.U


def off(got, ref):
    return ((R.f64(got) - ref).norm() / ref.norm()).item()


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("N", [4, 24, 40])
@pytest.mark.parametrize("lo,hi", [(1e-5, 1e-4), (1e-4, 1e-3), (1e-3, 4e-3)])
def test_slow_decays(lo, hi, N, cut):
    """d |A| from lo to hi, no input to the states: what is left of h0 behind T tokens, and of dh before them, is
    exp(A sum d). One block for each row walks all tokens, or sequences are cut into pieces."""
    T, C = 4096, 8
    B = 1 if cut else torch.cuda.get_device_properties(0).multi_processor_count
    r = torch.Generator().manual_seed(N)
    u = lambda *s: torch.rand(*s, generator=r)  # noqa: E731
    A = -(0.5 + u(C, N))                                            # 0.5 .. 1.5, each with steps of its channel
    d = (lo / 0.5) * (hi / lo / 3) ** u(B, T, C)                    # lo .. hi times the rate
    h0, dh = torch.randn(B, C, N, generator=r), torch.randn(B, C, N, generator=r)
    x, z = torch.randn(B, T, C, generator=r).cuda(), torch.zeros(B, T, 1, N).cuda()
    d, A, h0, dh = (v.cuda() for v in (d, A, h0, dh))
    h = torch.empty_like(h0)
    y, save = g.ssm_forward_save(x, d, A, z, z, softplus=False, h0=h0, h=h)
    dh0 = g.ssm_backward(x, d, A, z, z, torch.zeros_like(y), save, softplus=False, h0=h0, dh=dh)[-1]
    left = torch.exp(R.f64(d).sum(1)[..., None] * R.f64(A))
    assert off(h, R.f64(h0) * left) <= steps(T)
    assert off(dh0, R.f64(dh) * left) <= steps(T)


@pytest.mark.parametrize("N", [4, 24, 40])
def test_slow_decays_a_token_at_a_time(N):
    T, B, C = 1024, 3, 128
    r = torch.Generator().manual_seed(N)
    A = -(0.5 + torch.rand(C, N, generator=r)).cuda()
    d = (2e-4 * 20 ** torch.rand(T, B, C, generator=r)).cuda()
    h0 = torch.randn(B, C, N, generator=r).cuda()
    h, bc = h0.clone(), torch.zeros(B, 1, N, device="cuda")
    for t in range(T):
        g.ssm_step(d[t], d[t], A, bc, bc, h, softplus=False)
    assert off(h, R.f64(h0) * torch.exp(R.f64(d).sum(0)[..., None] * R.f64(A))) <= steps(T)


@pytest.mark.parametrize("N,G", [(16, 1), (24, 2), (64, 1)])
def test_norms_of_outputs(N, G):
    """Rates 1 .. N and steps log-uniform in 1e-3 .. 1e-1, as training starts from, over 577 tokens: states remember
    up to all of them, so the tokens' errors count as above; a step's softplus adds 12 u of d |A| for each token
    that is remembered, 12 u in all, gates, sums over states and the last rounding 8 u. A gradient is a
    product of two such quantities."""
    B, T, C = 1, 577, 66
    r = torch.Generator().manual_seed(N)
    n = lambda *s: torch.randn(*s, generator=r).cuda()  # noqa: E731
    size = torch.exp(torch.empty(C).uniform_(-6.9, -2.3, generator=r))
    x, dt, z, dy, Bm, Cm = n(B, T, C), 0.5 * n(B, T, C), n(B, T, C), n(B, T, C), n(B, T, G, N), n(B, T, G, N)
    A = -(torch.arange(1, N + 1) * (0.8 + 0.4 * torch.rand(C, N, generator=r))).cuda()
    D, bias, h0, dh = n(C), torch.log(torch.expm1(size)).cuda(), n(B, C, N), n(B, C, N)
    h = torch.empty_like(h0)
    kw = dict(D=D, z=z, dt_bias=bias, h0=h0)
    y, save = g.ssm_forward_save(x, dt, A, Bm, Cm, h=h, **kw)
    got = g.ssm_backward(x, dt, A, Bm, Cm, dy, save, dh=dh, **kw)
    ref = R.scan(x, dt, A, Bm, Cm, D, z, bias, True, None, h0, dy, dh)
    one = steps(T) + 20 * R.U
    bad = {k: v / one for k, v in (("y", off(y, ref["y"])), ("h", off(h, ref["h"]))) if not v <= one}
    for name, v in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0"), got):
        if not off(v, ref[name]) <= 2 * one:
            bad[name] = off(v, ref[name]) / one
    assert not bad, bad


def test_no_states_are_kept_without_gradients(monkeypatch):
    """Under no_grad the differentiable call is the plain one, though its parameters ask for gradients."""
    from linear_spatial_propagation_gspn_b200 import seq

    x, bc = torch.randn(2, 40, 32, device="cuda"), torch.randn(2, 40, 1, 16, device="cuda")
    A = (-torch.rand(32, 16, device="cuda")).requires_grad_(True)
    want = g.selective_scan(x, x, A, bc, bc)
    assert want.requires_grad
    monkeypatch.setattr(seq, "ssm_forward_save", lambda *a, **k: pytest.fail("states were kept"))
    with torch.no_grad():
        got = g.selective_scan(x, x, A, bc, bc)
    assert torch.equal(got, want) and not got.requires_grad
